// rows.cuh - attention of many query rows over paged latent rows (prompts, prompt chunks, shared
// prefixes), in the absorbed form the decode step uses:
//   S[r][t] = [q~ | q^R][r] . [c_j | k^R][t],  P = softmax over the keys row r may see,
//   O[r]    = sum_t P[r][t] c_j[t]
// A row r is one (query token, head) pair. Every head of a latent block reads the same cached rows,
// so the rows of a token's heads are stacked in one MMA tile: with 32 heads a block (MLRA-4) a tile
// of 128 rows is 4 tokens, and a prompt of any length fills its tiles to within 3 tokens. The key
// tile is also the value tile (its first d_b columns), so each cached byte is staged once.
//
// Work is split along one line: a unit is a token tile of one latent block (and head chunk), a
// unit's cost the key tiles it sees (plus a constant), and CTA c of the persistent grid takes the
// stretch [c * quota, (c + 1) * quota) of all the units' costs laid end to end. A unit that lies in
// one stretch is finished there; one that is cut leaves normalised fp32 partials with their
// log-sum-exp, merged afterwards in a fixed order. The split needs lengths that only the device
// has, so one block lays the units out in front of it: of the absorb kernel, or (per-head form) a
// kernel of one block.
//
// What bounds it: a 128 x 128 tile at d_b = 128, d_rope = 64 is 12 + 8 tcgen05 MMAs of 64 clocks
// (1280; the scores' MMAs, both operands from shared memory at N = 128, measure 85 each) against
// 16384 exponentials (1024 clocks of the special-function units), so two row tiles run in turn: one
// tile's softmax works while the other's MMAs run. Measured per pair of tiles: 3200 to 3300 clocks,
// of which the softmax of one tile takes 2800 and the MMAs of both 3060. This kernel alone: one step
// over a 32768-row prefix for 128 sequences of 128 heads (350 GFLOP) takes 290 us, 1.2 PFLOP/s; a
// 16384-token prompt (11.1 TFLOP) 8.5 ms, 1.3 PFLOP/s, with the clock at 1.6 GHz of 1.965 under the
// 1000 W power cap (the whole call 9.4 ms, 10.2 in long runs).
// Steps that got there, on that prompt as a whole call: one MMA warp and plan walks by every role 13.1
// ms; a walk warp, uniform-register MMA issue and the register split 10.3; separate issuers of scores
// and values with one score buffer in turn 9.7; masks and results in fewer instructions 9.35.
// Exponentials partly as polynomials on the multiply-add units measured slower (10.2 -> 10.3 to 11.1
// ms): the special-function units are not the bound.
#pragma once

#include "common.cuh"
#include "decode.cuh"
#include "proj.cuh"
#include "rowplan.cuh"

namespace mlra {

// One lane of a converged warp; the same one each time. The MMA warp runs its loops whole, and only
// the instructions that must come from one thread sit behind this predicate, so descriptors stay in
// uniform registers (with the loops themselves behind a lane test an MMA took 86 clocks to issue).
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// Shared-memory descriptors as two words (see smem_desc): the upper word is the same for all tiles of a
// layout, the lower one moves by offset / 16.
__host__ __device__ constexpr uint32_t desc_hi(uint32_t sbo, uint32_t layout) {
  return ((sbo >> 4) & 0x3FFFu) | (1u << 14) | (layout << 29);
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr >> 4) & 0x3FFFu) | (((lbo >> 4) & 0x3FFFu) << 16);
}
__device__ __forceinline__ void umma_ss(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A from tensor memory: its row r lies in lane r, two K elements a column.
__device__ __forceinline__ void umma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t b_hi,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
// A warpgroup's share of the block's registers (every warp of it executes this).
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// The largest of three; NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ void fma_f32x2(float& d0, float& d1, float a0, float a1, float b0, float b1, float c0,
                                          float c1) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(f2pack(a0, a1)), "l"(f2pack(b0, b1)), "l"(f2pack(c0, c1)));
  d0 = __uint_as_float(static_cast<uint32_t>(d));
  d1 = __uint_as_float(static_cast<uint32_t>(d >> 32));
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z,
                                            int w, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar)), "l"(policy)
      : "memory");
}

// ---------------------------------------------------------------------------------------
// The attention kernel
// ---------------------------------------------------------------------------------------
// DB, DR: block and RoPE widths; KT: keys a tile (64 or 128); DV: value columns a CTA keeps
// (DB, or a half of it where DB fp32 columns would fill the tensor memory); NQ row tiles in turn.
// A key tile is staged as its block columns (ring of CST) and its RoPE columns (ring of RST): the
// scores of both row tiles are formed early, after which the RoPE columns are done with, while the
// block columns wait for both P. At d_b = 128 that is what lets three tiles' block columns fit.
// Tensor memory: with two row tiles, one score buffer that they use in turn (a softmax warpgroup has
// it in registers about 200 clocks after it is ready, so the next scores are formed while the
// exponentials run) and a P buffer each; with one, two score buffers and one P buffer.
// Scores and values are issued by two warps: an MMA holds its issuer up while the tensor pipe's short
// queue is full, and each wait costs a few hundred clocks, which one warp's MMAs hide for the other.
// VST > 0: the per-head form. Keys and values are two buffers (a head's own, formed by the expansion
// kernel), so values have a ring of VST places of their own, and a tile's keys and RoPE columns are
// done with as soon as its scores are formed. A row tile is then 128 tokens of one head. The values
// are finite (see the expansion), so no tile is patched.
template <int DB_, int DR_, int KT_, int DV_, int NQ_, int CST_, int RST_, int VST_ = 0>
struct RowShape {
  static constexpr int DB = DB_, DR = DR_, KT = KT_, DV = DV_, NQ = NQ_, CST = CST_, RST = RST_,
                       VST = VST_;
  static constexpr bool SPLIT = VST > 0;
  static constexpr int HALVES = DB / DV;
  static constexpr int ROWS = 128 * NQ;     // query rows a unit
  static constexpr int CW = DB < 64 ? DB : 64, NC = DB / CW, C_ROWB = CW * 2;
  static constexpr int RW = DR < 64 ? DR : 64, NR = DR / RW, R_ROWB = RW * 2;
  static constexpr int QC_REG = 128 * C_ROWB, QR_REG = 128 * R_ROWB;
  static constexpr int Q_BYTES = NC * QC_REG + NR * QR_REG;
  static constexpr int KC_REG = KT * C_ROWB, KR_REG = KT * R_ROWB;
  static constexpr int C_BYTES = NC * KC_REG, R_BYTES = NR * KR_REG;
  static constexpr int V_BYTES = (DV / CW) * KC_REG;
  static constexpr int PST = SPLIT ? VST : CST;  // places of the ring that holds the values
  static constexpr int PAGE_TX = kPage * (DB + DR) * 2;
  static constexpr int SB = NQ == 1 ? 2 : 1;                  // score buffers
  static constexpr int S_COL = 0;
  static constexpr int P_COL = SB * KT;                       // KT / 2 columns a row tile
  static constexpr int O_COL = P_COL + NQ * (KT / 2);
  static constexpr int TMEM_USED = O_COL + NQ * DV;
  static constexpr int TMEM_COLS = TMEM_USED <= 128 ? 128 : TMEM_USED <= 256 ? 256 : 512;
  static constexpr int QK_WARP = 4 * NQ, PV_WARP = QK_WARP + 1, LOAD_WARP = QK_WARP + 2, FIX_WARP = QK_WARP + 3;
  static constexpr int THREADS = 32 * (FIX_WARP + 1);
  // Two row tiles: 384 threads are launched with 168 registers each (64,512); the two softmax
  // warpgroups take 208 (53,248) and the other one keeps 88 (11,264).
  static constexpr bool REGS = NQ == 2;
  static constexpr int PARTS = 4;            // unit parts handed out ahead
  static constexpr int READERS = 4 * NQ + 4; // warps that read them
  static constexpr int NBARS = 4 * CST + RST + 2 * VST + 2 * NQ + 4 + 3 * NQ + 2 + 2 * PARTS;
  static constexpr int OFF_C = NQ * Q_BYTES;
  static constexpr int OFF_R = OFF_C + CST * C_BYTES;
  static constexpr int OFF_V = OFF_R + RST * R_BYTES;
  static constexpr int OFF_BAR = OFF_V + VST * V_BYTES;
  static constexpr int OFF_PARTS = (OFF_BAR + NBARS * 8 + 15) / 16 * 16;
  static constexpr int SMEM = OFF_PARTS + PARTS * 48 + 64 + 1024;
  static_assert(SMEM <= 227 * 1024 && TMEM_USED <= 512, "shared and tensor memory of one CTA");
  static_assert(KT == 64 || KT == 128, "whole pages");
  static_assert(DV <= 256 && DV % 16 == 0 && DB % DV == 0, "one PV instruction's columns");
  static_assert(Q_BYTES % 1024 == 0 && C_BYTES % 1024 == 0 && R_BYTES % 1024 == 0 && KC_REG % 1024 == 0 &&
                    QC_REG % 1024 == 0 && KR_REG % 1024 == 0 && QR_REG % 1024 == 0,
                "swizzled regions start on 1024 bytes");
  static_assert(!SPLIT || (HALVES == 1 && RST == CST && VST <= CST), "per-head form");
  static_assert(RST <= CST && (NQ == 1 || CST >= 2), "a tile's full barrier counts both rings");
};

struct RowParams {
  RowPlan plan;
  const int* page_table;   // null: page i of sequence b is b * pt_stride + i
  int pt_stride, num_pages;
  // the first `own` sequences of the plan have pages of another table, and their results come behind
  // the others' (o_f32, lse: [own] tokens more)
  const int* own_table;
  int own_stride, own;
  int causal;
  int nsub;                // (latent block, head chunk) pairs
  int chunks;              // head chunks of a block
  int heads_tile;          // heads of a row tile's tokens: min(heads of a block, np)
  int tok_tile;            // tokens of a row tile: 128 / heads_tile
  int heads_block, vh;     // heads of a block, (virtual) heads in all
  int d_c;
  float s_scale;           // from a score (packed query times staged row) to log2 units
  float o_scale;           // value of a staged latent element (1, or the E4M3 cache's scale)
  int seq_rows, kv_rows;   // per-head form: rows a sequence and a head have in the key / value buffer
  __nv_bfloat16* o_bf16;   // [tokens][vh][DB], or null
  float* o_f32;            // [tokens][vh][DB] when o_bf16 is null
  float* lse;              // [tokens][vh] or null
  float lse_mul;           // from log2 to what lse holds
  float* part_o;           // [2 * CTAs][ROWS][DV]
  float* part_lse;         // [2 * CTAs][ROWS] log2
  int* status;
  EarlyTags tags;
  unsigned long long wait_limit_ns;
};

// Four lanes that hold four 16-byte pieces of their own rows each exchange them, so that lane j ends
// with piece j of all four rows: a store then covers 64 bytes in a row instead of 16.
__device__ __forceinline__ void exchange4(uint4 (&v)[4], int lane) {
  uint32_t* w = reinterpret_cast<uint32_t*>(v);
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      if (p & o) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = w[p * 4 + e], b = w[(p | o) * 4 + e];
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? a : b, o);
        w[p * 4 + e] = up ? got : a;
        w[(p | o) * 4 + e] = up ? b : got;
      }
    }
  }
}

// A unit cut by the stretches leaves CTA c's part in slot 2c + 1 where the part begins the unit,
// in slot 2c where it goes on with one begun before (a stretch holds at most one of each).
template <class Sh>
__global__ void __launch_bounds__(Sh::THREADS, 1)
    mlra_rows_kernel(const __grid_constant__ CUtensorMap map_c, const __grid_constant__ CUtensorMap map_r,
                     const __grid_constant__ CUtensorMap map_qc, const __grid_constant__ CUtensorMap map_qr,
                     const RowParams p) {
  constexpr int NQ = Sh::NQ, KT = Sh::KT, CST = Sh::CST, RST = Sh::RST, VST = Sh::VST, PST = Sh::PST, DV = Sh::DV;
  constexpr bool SPLIT = Sh::SPLIT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* qbuf = smem;
  uint8_t* cring = smem + Sh::OFF_C;
  uint8_t* rring = smem + Sh::OFF_R;
  uint8_t* vring = smem + (SPLIT ? Sh::OFF_V : Sh::OFF_C);  // the values
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + Sh::OFF_BAR);  // [CST] a key tile has landed
  uint64_t* cempty = kfull + CST;        // [CST] its block columns are done with
  uint64_t* rempty = cempty + CST;       // [RST] its RoPE columns are
  uint64_t* qfull = rempty + RST;        // [NQ]
  uint64_t* qempty = qfull + NQ;         // [NQ]
  // (two row tiles: index q; one: the score buffer, alternating)
  uint64_t* sfull = qempty + NQ;         // [2] scores are there
  uint64_t* sfree = sfull + 2;           // [2] and have been read into registers
  uint64_t* pfull = sfree + 2;           // [NQ] P is there
  uint64_t* pvdone = pfull + NQ;         // [NQ] P has been read, O is up to date
  uint64_t* ofree = pvdone + NQ;         // [NQ] a part's O has been read
  // (one a ring place: scores run ahead of values, so several tiles may wait for their patch)
  uint64_t* patch = ofree + NQ;          // [CST] a key tile is ready to be patched
  uint64_t* patched = patch + CST;       // [CST] and has been
  uint64_t* drained = patched + CST;     // [2]
  uint64_t* vfull = drained + 2;         // [VST] per-head form: values have landed
  uint64_t* vempty = vfull + VST;        // [VST] and are done with
  uint64_t* pready = vempty + VST;        // [PARTS]
  uint64_t* pread = pready + Sh::PARTS;  // [PARTS]
  int4* parts = reinterpret_cast<int4*>(smem + Sh::OFF_PARTS);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(parts + 3 * Sh::PARTS);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* drain_err = abort_flag + 1;

  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    for (int s = 0; s < CST; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&cempty[s], 1);
      mbar_init(&patch[s], 1);
      mbar_init(&patched[s], 1);
    }
    for (int s = 0; s < VST; ++s) {
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 1);
    }
    for (int s = 0; s < RST; ++s) mbar_init(&rempty[s], 1);
    for (int q = 0; q < 2; ++q) {
      mbar_init(&sfull[q], 1);
      mbar_init(&sfree[q], 4);
      mbar_init(&drained[q], 1);
    }
    for (int q = 0; q < NQ; ++q) {
      mbar_init(&qfull[q], 1);
      mbar_init(&qempty[q], 1);
      mbar_init(&pfull[q], 4);
      mbar_init(&pvdone[q], 1);
      mbar_init(&ofree[q], 4);
    }
    for (int i = 0; i < Sh::PARTS; ++i) {
      mbar_init(&pready[i], 1);
      mbar_init(&pread[i], Sh::READERS);
    }
    *abort_flag = 0;
    *drain_err = 0;
    fence_mbar_init();
  }
  if (warp == Sh::LOAD_WARP && lane == 0) {
    tma_prefetch_map(&map_c);
    tma_prefetch_map(&map_r);
    tma_prefetch_map(&map_qc);
    tma_prefetch_map(&map_qr);
  }
  // The plan, the packed query and the cleared status word come from kernels before this one. The
  // tensor memory is taken after them too, so no CTA that waits holds what an earlier one needs.
  grid_dependency_wait();
  if (warp == Sh::QK_WARP) {
    tmem_alloc(tmem_slot, Sh::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  grid_launch_dependents();

  uint32_t kt = 0;    // key tiles so far (rings)
  uint32_t uc = 0;    // unit parts so far
  uint32_t fixes = 0; // parity of the patches so far, a bit a ring place
  auto wait = [&](uint64_t* b, uint32_t par) {
    return __all_sync(0xffffffffu, mbar_wait(b, par, abort_flag, p.wait_limit_ns));
  };
  // the next unit part from the walk warp's ring; false after the last one
  auto take = [&](UnitPart& u) {
    const int e = uc % Sh::PARTS;
    u.valid = false;
    if (!wait(&pready[e], (uc / Sh::PARTS) & 1)) return false;
    const int4 a = parts[3 * e], b = parts[3 * e + 1];
    u.valid = parts[3 * e + 2].x != 0;
    u.t = {a.x, a.y, a.z, a.w};
    u.sub = b.x; u.kv = b.y; u.begin = b.z; u.end = b.w;
    __syncwarp();
    if (lane == 0) mbar_arrive(&pread[e]);
    ++uc;
    return u.valid;
  };
  // row tiles a unit part uses
  auto rows_of = [&](const UnitPart& x) { return NQ == 2 && x.t.ntok > p.tok_tile ? 2 : 1; };
  // key tiles of the part that row tile q sees any of: the first row tile's tokens may all lie before
  // the part's last key tiles, which are then formed for the second one alone
  auto tiles_of_row = [&](const UnitPart& x, int q) {
    const int last = min(x.t.ntok, (q + 1) * p.tok_tile) - 1;
    const int lim = max(p.causal ? x.t.lim0 + last : x.t.lim0, 0);
    return max(min(x.end, (lim + KT - 1) / KT) - x.begin, 0);
  };
  UnitPart u;
  // (the register split sits in the two branches, so that each is compiled for its own share)
  if (warp >= 4 * NQ) {
    if constexpr (Sh::REGS) regs_down<88>();
    if (warp == Sh::LOAD_WARP) {
      // ------------------------------ TMA loads ------------------------------
      const uint64_t pol = l2_policy_evict_last();
      uint32_t issued = 0, parity = 0;     // key tiles' full barriers
      uint32_t q_issued = 0, q_parity = 0; // query barriers
      uint32_t v_issued = 0, v_parity = 0; // values' full barriers
      uint32_t qc[NQ];                     // query loads so far, a row tile
#pragma unroll
      for (int q = 0; q < NQ; ++q) qc[q] = 0;
      // the part's queries (behind its first key tile, whose place is free earlier); one lane
      auto load_queries = [&](const UnitPart& x) {
        const int rows = p.heads_tile * p.tok_tile, sub = x.sub / Sh::HALVES, nrow = rows_of(x);
        for (int q = 0; q < nrow; ++q) {
          if (!mbar_wait(&qempty[q], (qc[q] & 1) ^ 1, abort_flag, p.wait_limit_ns)) return false;
          mbar_arrive_expect_tx(&qfull[q], rows * (Sh::DB + Sh::DR) * 2);
          q_issued |= 1u << q;
          q_parity = (q_parity & ~(1u << q)) | ((qc[q] & 1) << q);
          ++qc[q];
          uint8_t* dst = qbuf + q * Sh::Q_BYTES;
          const int tok = x.t.tok0 + q * p.tok_tile;
          for (int r = 0; r < Sh::NC; ++r)
            tma_load_4d(dst + r * Sh::QC_REG, &map_qc, &qfull[q], r * Sh::CW, 0, sub, tok, pol);
          for (int r = 0; r < Sh::NR; ++r)
            tma_load_4d(dst + Sh::NC * Sh::QC_REG + r * Sh::QR_REG, &map_qr, &qfull[q], Sh::DB + r * Sh::RW, 0, sub,
                        tok, pol);
        }
        return true;
      };
      auto note = [&](uint32_t& mask, uint32_t& par, int s, uint32_t ph) {
        mask |= 1u << s;
        par = (par & ~(1u << s)) | (ph << s);
      };
      bool ok = true;
      if constexpr (SPLIT) {
        // Keys go a tile ahead of values, whose place comes free later, and a part's first keys and its
        // queries ahead of the last values of the part before.
        auto load_keys = [&](const UnitPart& x, int t, uint32_t n) {
          const int s = n % CST, r0 = x.t.b * p.seq_rows + t * KT, y = x.sub * p.kv_rows + r0;
          const uint32_t ph = (n / CST) & 1;
          if (!mbar_wait(&cempty[s], ph ^ 1, abort_flag, p.wait_limit_ns)) return false;
          mbar_arrive_expect_tx(&kfull[s], Sh::C_BYTES + Sh::R_BYTES);
          note(issued, parity, s, ph);
          for (int r = 0; r < Sh::NC; ++r)
            tma_load_2d(cring + s * Sh::C_BYTES + r * Sh::KC_REG, &map_c, &kfull[s], r * Sh::CW, y, pol);
          for (int r = 0; r < Sh::NR; ++r)
            tma_load_2d(rring + s * Sh::R_BYTES + r * Sh::KR_REG, &map_r, &kfull[s], r * Sh::RW, r0, pol);
          return true;
        };
        UnitPart v;
        bool more = take(u);
        if (more && lane == 0) ok = load_keys(u, u.begin, 0) && load_queries(u);
        while (more && __shfl_sync(0xffffffffu, ok, 0)) {
          bool next = false;
          for (int t = u.begin; t < u.end; ++t, ++kt) {
            const bool last = t + 1 == u.end;
            if (last) next = take(v);
            if (lane == 0 && ok) {
              if (!last) ok = load_keys(u, t + 1, kt + 1);
              else if (next) ok = load_keys(v, v.begin, kt + 1) && load_queries(v);
              const int s = kt % PST;
              const uint32_t ph = (kt / PST) & 1;
              ok = ok && mbar_wait(&vempty[s], ph ^ 1, abort_flag, p.wait_limit_ns);
              if (ok) {
                mbar_arrive_expect_tx(&vfull[s], Sh::V_BYTES);
                note(v_issued, v_parity, s, ph);
                for (int r = 0; r < DV / Sh::CW; ++r)
                  tma_load_2d(vring + s * Sh::V_BYTES + r * Sh::KC_REG, &map_c, &vfull[s], Sh::DB + r * Sh::CW,
                              u.sub * p.kv_rows + u.t.b * p.seq_rows + t * KT, pol);
              }
            }
          }
          u = v;
          more = next;
        }
      }
      while (!SPLIT && ok && take(u)) {
        const int sub = u.sub / Sh::HALVES;
        const int blk = sub / p.chunks;
        const int pages = (tile_limit(u.t, p.causal) + kPage - 1) / kPage;
        const bool own = u.t.b < p.own;
        const size_t row = own ? (size_t)u.t.b * p.own_stride : (size_t)(u.t.b - p.own) * p.pt_stride;
        const int* table = own ? p.own_table : p.page_table;
        constexpr int PPT = KT / kPage;  // pages a key tile
        int wb = u.begin * PPT;
        // page ids come through a window of two registers a lane, the next 32 read ahead
        auto ids = [&](int base) {
          const int pg = base + lane;
          if (pg >= pages) return 0;
          return table != nullptr ? __ldg(table + row + pg) : (int)row + pg;
        };
        int w0 = ids(wb), w1 = ids(wb + 32);
        for (int t = u.begin; t < u.end && ok; ++t, ++kt) {
          const int p0 = t * PPT;
          if (p0 >= wb + 32) {
            wb += 32;
            w0 = w1;
            w1 = ids(wb + 32);
          }
          int id[PPT];
#pragma unroll
          for (int x = 0; x < PPT; ++x) id[x] = __shfl_sync(0xffffffffu, w0, (p0 + x - wb) & 31);
          const int npg = min(PPT, pages - p0);
          if (lane == 0) {
            const int s = kt % CST, rs = kt % RST;
            const uint32_t ph = (kt / CST) & 1;
            ok = mbar_wait(&cempty[s], ph ^ 1, abort_flag, p.wait_limit_ns) &&
                 mbar_wait(&rempty[rs], ((kt / RST) & 1) ^ 1, abort_flag, p.wait_limit_ns);
            if (ok) {
              mbar_arrive_expect_tx(&kfull[s], npg * Sh::PAGE_TX);
              note(issued, parity, s, ph);
#pragma unroll
              for (int x = 0; x < PPT; ++x) {
                if (x >= npg) break;
                if (id[x] < 0 || id[x] >= p.num_pages) {
                  set_status(p.status, kErrPageOob);
                  id[x] = 0;
                }
                const int y = id[x] * kPage;
                for (int r = 0; r < Sh::NC; ++r)
                  tma_load_2d(cring + s * Sh::C_BYTES + r * Sh::KC_REG + x * kPage * Sh::C_ROWB, &map_c, &kfull[s],
                              blk * Sh::DB + r * Sh::CW, y, pol);
                for (int r = 0; r < Sh::NR; ++r)
                  tma_load_2d(rring + rs * Sh::R_BYTES + r * Sh::KR_REG + x * kPage * Sh::R_ROWB, &map_r, &kfull[s],
                              p.d_c + r * Sh::RW, y, pol);
              }
            }
            if (t == u.begin) ok = ok && load_queries(u);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
        }
      }
      if (lane == 0) {
        // nothing may still be landing when the CTA's shared memory is released
        for (int s = 0; s < CST; ++s)
          if ((issued >> s) & 1)
            if (!mbar_wait_drain(&kfull[s], (parity >> s) & 1, p.wait_limit_ns)) *drain_err = 1;
        for (int q = 0; q < NQ; ++q)
          if ((q_issued >> q) & 1)
            if (!mbar_wait_drain(&qfull[q], (q_parity >> q) & 1, p.wait_limit_ns)) *drain_err = 1;
        for (int s = 0; s < VST; ++s)
          if ((v_issued >> s) & 1)
            if (!mbar_wait_drain(&vfull[s], (v_parity >> s) & 1, p.wait_limit_ns)) *drain_err = 1;
      }
    } else if (warp == Sh::QK_WARP) {
      // ------------------------------ scores ------------------------------
      const bool one = elect_lane();
      constexpr uint32_t idesc_qk = idesc_bf16_f32(128, KT, false, false);
      constexpr uint32_t c_hi = desc_hi(8 * Sh::C_ROWB, swizzle_code(Sh::C_ROWB));
      constexpr uint32_t r_hi = desc_hi(8 * Sh::R_ROWB, swizzle_code(Sh::R_ROWB));
      const uint32_t q_lo = desc_lo(smem_u32(qbuf), 16), c_lo = desc_lo(smem_u32(cring), 16);
      const uint32_t r_lo = desc_lo(smem_u32(rring), 16);
      uint32_t sc[NQ], qc[NQ];  // score tiles and queries so far
#pragma unroll
      for (int q = 0; q < NQ; ++q) sc[q] = qc[q] = 0;
      int last = -1;            // two row tiles: whose scores the buffer holds
      bool ok = true;
      while (ok && take(u)) {
        const int n = u.end - u.begin, nrow = rows_of(u), n0 = tiles_of_row(u, 0);
        if (n0 == 0) {
          // a part whose first row tile sees none of it: its query is given back unread
          ok = wait(&qfull[0], qc[0] & 1);
          ++qc[0];
          if (one) umma_commit(&qempty[0]);
        }
        for (int i = 0; i < n && ok; ++i, ++kt) {
          ok = wait(&kfull[kt % CST], (kt / CST) & 1);
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if (q >= nrow || !ok) break;
            if (NQ == 2 && q == 0 && i >= n0) continue;
            if (i == 0) {
              ok = wait(&qfull[q], qc[q] & 1);
              ++qc[q];
            }
            // the score buffer's last contents are in registers
            if (NQ == 1) {
              if (kt >= 2) ok = ok && wait(&sfree[kt & 1], ((kt >> 1) - 1) & 1);
            } else if (last >= 0) {
              ok = ok && (last == 0 ? wait(&sfree[0], (sc[0] - 1) & 1) : wait(&sfree[1], (sc[NQ - 1] - 1) & 1));
            }
            if (!ok) break;
            last = q;
            ++sc[q];
            tc_fence_after();
            const uint32_t a0 = q_lo + q * (Sh::Q_BYTES >> 4), b0 = c_lo + (kt % CST) * (Sh::C_BYTES >> 4);
            const uint32_t b1 = r_lo + (kt % RST) * (Sh::R_BYTES >> 4);
            const uint32_t d = tbase + Sh::S_COL + (NQ == 1 ? (kt & 1) * KT : 0);
            if (one) {
#pragma unroll
              for (int r = 0; r < Sh::NC; ++r)
#pragma unroll
                for (int ks = 0; ks < Sh::C_ROWB / 32; ++ks)
                  umma_ss(d, a0 + ((r * Sh::QC_REG + ks * 32) >> 4), c_hi, b0 + ((r * Sh::KC_REG + ks * 32) >> 4), c_hi,
                          idesc_qk, (r > 0 || ks > 0) ? 1u : 0u);
#pragma unroll
              for (int r = 0; r < Sh::NR; ++r)
#pragma unroll
                for (int ks = 0; ks < Sh::R_ROWB / 32; ++ks)
                  umma_ss(d, a0 + ((Sh::NC * Sh::QC_REG + r * Sh::QR_REG + ks * 32) >> 4), r_hi,
                          b1 + ((r * Sh::KR_REG + ks * 32) >> 4), r_hi, idesc_qk, 1u);
              umma_commit(&sfull[NQ == 1 ? kt & 1 : q]);
              if (i == (q == 0 ? n0 : n) - 1) umma_commit(&qempty[q]);
              if (q == nrow - 1) {
                umma_commit(SPLIT ? &cempty[kt % CST] : &rempty[kt % RST]);
                // a tile that reaches past what the part's first token sees is patched (see the patch
                // warp) between its score MMAs and its value MMAs
                if (!SPLIT && (u.begin + i + 1) * KT > u.t.lim0) umma_commit(&patch[kt % PST]);
              }
            }
          }
        }
      }
      if (one) umma_commit(&drained[0]);
      if (!mbar_wait_drain(&drained[0], 0, p.wait_limit_ns)) *drain_err = 1;
      __syncwarp();
    } else if (warp == Sh::PV_WARP) {
      // ------------------------------ values ------------------------------
      const bool one = elect_lane();
      constexpr uint32_t idesc_pv = idesc_bf16_f32(128, DV, false, true);
      constexpr uint32_t c_hi = desc_hi(8 * Sh::C_ROWB, swizzle_code(Sh::C_ROWB));
      const uint32_t v_lo = desc_lo(smem_u32(vring), Sh::KC_REG);
      constexpr uint32_t place = (SPLIT ? Sh::V_BYTES : Sh::C_BYTES) >> 4;
      uint32_t pc[NQ], oc[NQ];  // P tiles and parts so far
#pragma unroll
      for (int q = 0; q < NQ; ++q) pc[q] = oc[q] = 0;
      bool ok = true;
      while (ok && take(u)) {
        const int n = u.end - u.begin, nrow = rows_of(u), n0 = tiles_of_row(u, 0);
        const uint32_t half = (u.sub % Sh::HALVES) * ((DV / Sh::CW) * (Sh::KC_REG >> 4));
        for (int i = 0; i < n && ok; ++i, ++kt) {
          if constexpr (SPLIT) ok = wait(&vfull[kt % PST], (kt / PST) & 1);
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if (q >= nrow || !ok) break;
            if (NQ == 2 && q == 0 && i >= n0) continue;
            ok = wait(&pfull[q], pc[q] & 1);
            ++pc[q];
            // (the tile's first reader waits for its patch)
            if (!SPLIT && q == (NQ == 2 && i >= n0 ? 1 : 0) && (u.begin + i + 1) * KT > u.t.lim0) {
              ok = ok && wait(&patched[kt % PST], (fixes >> (kt % PST)) & 1);
              fixes ^= 1u << (kt % PST);
            }
            if (i == 0) {
              ok = ok && wait(&ofree[q], (oc[q] & 1) ^ 1);
              ++oc[q];
            }
            if (!ok) break;
            tc_fence_after();
            const uint32_t b0 = v_lo + (kt % PST) * place + half;
            const uint32_t a = tbase + Sh::P_COL + q * (KT / 2);
            if (one) {
#pragma unroll
              for (int ks = 0; ks < KT / 16; ++ks)
                umma_ts(tbase + Sh::O_COL + q * DV, a + ks * 8, b0 + ((ks * 16 * Sh::C_ROWB) >> 4), c_hi, idesc_pv,
                        (i > 0 || ks > 0) ? 1u : 0u);
              umma_commit(&pvdone[q]);
              // (every score of the tile was formed before the last row tile's P)
              if (q == nrow - 1) umma_commit(SPLIT ? &vempty[kt % PST] : &cempty[kt % PST]);
            }
          }
        }
      }
      if (one) umma_commit(&drained[1]);
      if (!mbar_wait_drain(&drained[1], 0, p.wait_limit_ns)) *drain_err = 1;
      __syncwarp();
    } else if (warp == Sh::FIX_WARP) {
      // ------------------------------ patches ------------------------------
      // A masked key has P = 0, but 0 x NaN is NaN: where a key tile reaches past what the unit's
      // first token sees, the value rows no token of the unit sees are zeroed (they may lie past the
      // sequence's end, where a slot may hold anything), and elements of the rows that only some of
      // its tokens see are zeroed where they are not finite. A token that does see such a row gets
      // its NaN through the score, whose MMA has read the tile before it is patched.
      // This warp also walks the plan and hands the unit parts out, two ahead of the one it is at.
      const int4 h1 = __ldg(reinterpret_cast<const int4*>(p.plan.hdr) + 1);
      const int tiles = __ldg(p.plan.hdr);
      UnitWalk walk;
      Stretch st;
      st.quota = join64(h1.x, h1.y);
      st.lo = min((long long)blockIdx.x * st.quota, join64(h1.z, h1.w));
      st.hi = min(st.lo + st.quota, join64(h1.z, h1.w));
      // Per-head form, many units: whole ones in turn, so that the CTAs work on a few heads of one
      // sequence at a time, whose keys and values L2 holds (with stretches each streams its own from
      // memory: 30 GB read for one 16384-token prompt of 128 heads, 11.1 ms)
      const bool whole_units = SPLIT && tiles * p.nsub >= 8 * (int)gridDim.x;
      if (whole_units) walk.init_whole(&p.plan, tiles, blockIdx.x, gridDim.x, p.nsub, KT, p.causal);
      else walk.init(&p.plan, tiles, st, blockIdx.x, p.nsub * Sh::HALVES, KT, p.causal);
      uint32_t given = 0;
      bool more = true;
      auto give = [&]() {
        const UnitPart g = whole_units ? walk.next_whole() : walk.next();
        const int e = given % Sh::PARTS;
        if (!wait(&pread[e], ((given / Sh::PARTS) & 1) ^ 1)) return false;
        if (lane == 0) {
          parts[3 * e] = make_int4(g.t.b, g.t.tok0, g.t.ntok, g.t.lim0);
          parts[3 * e + 1] = make_int4(g.sub, g.kv, g.begin, g.end);
          parts[3 * e + 2].x = g.valid;
          mbar_arrive(&pready[e]);
        }
        if (given == 0 && lane == 0) {
          // for the merge: the unit that this stretch goes on with, and the CTAs that share it
          int c0 = -1, c1 = -1;
          if (g.valid && g.begin > 0) {
            const long long first = walk.at + (long long)g.sub * unit_cost(g.kv) + kUnitCost;
            c0 = (int)(first / st.quota);
            c1 = (int)((first + g.kv - 1) / st.quota);
          }
          p.plan.cut[2 * blockIdx.x] = make_int4(c0, c1, g.sub, 0);
          p.plan.cut[2 * blockIdx.x + 1] = make_int4(g.t.tok0, g.t.ntok, 0, 0);
        }
        __syncwarp();
        ++given;
        more = g.valid;
        return true;
      };
      bool ok = give();
      if (ok && more) ok = give();
      while (ok && take(u)) {
        if (more) ok = give();
        if (!ok) break;
        const int lim = tile_limit(u.t, p.causal);
        for (int t = u.begin; t < u.end && ok; ++t, ++kt) {
          if (SPLIT || (t + 1) * KT <= u.t.lim0) continue;
          // the MMAs that form this key tile's scores have read it (and it had landed)
          ok = wait(&patch[kt % PST], (fixes >> (kt % PST)) & 1) && wait(&kfull[kt % PST], (kt / PST) & 1);
          if (!ok) break;
          fixes ^= 1u << (kt % PST);
          uint8_t* st_mem = cring + (kt % PST) * Sh::C_BYTES;
          const int k0 = t * KT;
          const int some = max(0, min(KT, max(u.t.lim0, 0) - k0));  // rows [some, none) only some tokens see
          const int none = max(0, min(KT, lim - k0));
          constexpr int CPR = Sh::C_ROWB / 16, REGS = Sh::NC;
          for (int r = 0; r < REGS; ++r)
#pragma unroll 4
            for (int i = none * CPR + lane; i < KT * CPR; i += 32)
              *reinterpret_cast<uint4*>(st_mem + r * Sh::KC_REG + i * 16) = make_uint4(0, 0, 0, 0);
          // 0 x value sums to NaN where any is not finite (rare): one multiply-add a pair, and eight
          // loads under way, for up to 32 KB
          const __nv_bfloat162 zero = __floats2bfloat162_rn(0.f, 0.f);
          __nv_bfloat162 acc[4] = {zero, zero, zero, zero};
          for (int r = 0; r < REGS; ++r)
#pragma unroll 8
            for (int i = some * CPR + lane; i < none * CPR; i += 32) {
              const uint4 x = *reinterpret_cast<const uint4*>(st_mem + r * Sh::KC_REG + i * 16);
              const __nv_bfloat162* h2 = reinterpret_cast<const __nv_bfloat162*>(&x);
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[e] = __hfma2(h2[e], zero, acc[e]);
            }
          const float2 bad = __bfloat1622float2(__hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3])));
          if (__any_sync(0xffffffffu, bad.x != 0.f || bad.y != 0.f)) {  // NaN != 0
            for (int r = 0; r < REGS; ++r)
              for (int i = some * CPR + lane; i < none * CPR; i += 32) {
                uint4* at = reinterpret_cast<uint4*>(st_mem + r * Sh::KC_REG + i * 16);
                uint4 x = *at;
                uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
                  if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0x0000ffffu;
                }
                *at = x;
              }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&patched[kt % PST]);
        }
      }
    }
  } else {
    if constexpr (Sh::REGS) regs_up<208>();
    // ------------------------------ softmax and results ------------------------------
    // A thread owns one row. The running maximum is raised only when a score passes it by more
    // than 8 (log2 units), so P stays below 2^8 and O is rescaled in tensor memory only then.
    const int q = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int tl = row / p.heads_tile;                     // token within the row tile
    const int hr = row - tl * p.heads_tile;                // head within the tile's heads
    const int tok = q * p.tok_tile + tl;                   // token within the unit
    const bool row_in = tl < p.tok_tile;
    const uint32_t o_addr = tbase + lane_base + Sh::O_COL + q * DV;
    // the four rows this lane stores a piece of (see exchange4): their tokens and places in a part
    int tok4[4], off4[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int rr = (row & ~3) + r, t4 = rr / p.heads_tile;
      tok4[r] = t4 < p.tok_tile ? q * p.tok_tile + t4 : 0x7fffffff;
      off4[r] = ((q * p.tok_tile + t4) * p.vh + (rr - t4 * p.heads_tile)) * Sh::DB + (lane & 3) * 8;
    }
    uint32_t sc = 0;                                       // score tiles so far
    bool ok = true;
    const float sc_mul = p.s_scale, slack = 8.f / sc_mul;
    while (ok && take(u)) {
      if (q >= rows_of(u)) continue;
      const int n = tiles_of_row(u, q);
      const int lim = p.causal ? u.t.lim0 + tok : u.t.lim0;  // keys this row sees
      float m = -INFINITY, l = 0.f;
      for (int i = 0; i < n; ++i, ++sc) {
        ok = NQ == 1 ? wait(&sfull[sc & 1], (sc >> 1) & 1) : wait(&sfull[q], sc & 1);
        if (!ok) break;
        tc_fence_after();
        const uint32_t s_addr = tbase + lane_base + Sh::S_COL + (NQ == 1 ? (sc & 1) * KT : 0);
        const uint32_t p_addr = tbase + lane_base + Sh::P_COL + q * (KT / 2);
        float s[KT];
        tmem_load_row<KT>(s_addr, s);
        tmem_ld_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sfree[NQ == 1 ? sc & 1 : q]);
        const int k0 = (u.begin + i) * KT;
        if (k0 + KT > u.t.lim0) {
          // 16 keys at a time: those every row of the warp sees are left alone
          const int seen = lim - k0, all = __reduce_min_sync(0xffffffffu, seen);
#pragma unroll
          for (int c0 = 0; c0 < KT; c0 += 16) {
            if (all >= c0 + 16) continue;
#pragma unroll
            for (int c = c0; c < c0 + 16; ++c) s[c] = c < seen ? s[c] : -INFINITY;
          }
        }
        float x0 = s[0], x1 = s[1], x2 = s[2], x3 = s[3];
#pragma unroll
        for (int c = 4; c + 8 <= KT; c += 8) {
          x0 = max3_nan(x0, s[c], s[c + 1]);
          x1 = max3_nan(x1, s[c + 2], s[c + 3]);
          x2 = max3_nan(x2, s[c + 4], s[c + 5]);
          x3 = max3_nan(x3, s[c + 6], s[c + 7]);
        }
        x0 = max3_nan(x0, s[KT - 4], s[KT - 3]);
        x1 = max3_nan(x1, s[KT - 2], s[KT - 1]);
        const float mt = max3_nan(max3_nan(x0, x1, x2), x3, x3);
        // P's place is free and O holds the sums up to the tile before
        if (sc > 0) ok = wait(&pvdone[q], (sc - 1) & 1);
        if (!ok) break;
        if (i == 0) {
          m = mt;
        } else {
          const bool raise = mt > m + slack;
          if (__any_sync(0xffffffffu, raise)) {
            tc_fence_after();
            const float a = raise ? fast_exp2((m - mt) * sc_mul) : 1.f;
            l *= a;
            if (raise) m = mt;
#pragma unroll 1
            for (int c = 0; c < DV; c += 32) {
              float o[32];
              tmem_load_row<32>(o_addr + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] *= a;
              tmem_store_row<32>(o_addr + c, o);
            }
            tmem_st_wait();
          }
        }
        const float mu = m == -INFINITY ? 0.f : -m * sc_mul;  // a row that sees no key of this part: P = 0
        float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
        for (int c0 = 0; c0 < KT; c0 += 64) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 64; c += 2) {
            float e0, e1;
            fma_f32x2(e0, e1, s[c0 + c], s[c0 + c + 1], sc_mul, sc_mul, mu, mu);
            e0 = fast_exp2(e0);
            e1 = fast_exp2(e1);
            if (c & 2) add_f32x2(l2, l3, l2, l3, e0, e1);
            else add_f32x2(l0, l1, l0, l1, e0, e1);
            pk[c / 2] = pack_bf16x2(e0, e1);  // P to bf16 (half a step 2^-8 relative) for the tensor core
          }
          tmem_st32(p_addr + c0 / 2, pk);
        }
        l += (l0 + l1) + (l2 + l3);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[q]);
      }
      if (!ok) break;
      if (n > 0) ok = wait(&pvdone[q], (sc - 1) & 1);
      if (!ok) break;
      tc_fence_after();
      // ---- results of this part ----
      const int half = u.sub % Sh::HALVES, sub = u.sub / Sh::HALVES;
      const int head0 = (sub / p.chunks) * p.heads_block + (sub % p.chunks) * p.heads_tile;
      const bool mine = row_in && tok < u.t.ntok;
      const bool whole = u.begin == 0 && u.end == u.kv;
      const int slot = 2 * blockIdx.x + (u.begin == 0 ? 1 : 0);
      const float inv = l > 0.f ? p.o_scale / l : (l == 0.f ? 0.f : l);  // NaN stays NaN
      const float lse2 = l == 0.f ? -INFINITY : m * sc_mul + __log2f(l);
      const int tok_out = u.t.tok0 + (u.t.b < p.own ? p.own : 0);
      const size_t at = (size_t)(tok_out + tok) * p.vh + head0 + hr;
      const size_t pat = (size_t)slot * Sh::ROWS + q * 128 + row;
      if (mine) {
        // (column halves are cut on their own: the one that is whole writes its lse even where the other
        // is not; where both are, they write the same bits, having formed the same scores)
        if (!whole)
          p.part_lse[pat] = lse2;
        else if (p.lse != nullptr)
          p.lse[at] = lse2 * p.lse_mul;
      }
      __nv_bfloat16* const out = p.o_bf16 + ((size_t)tok_out * p.vh + head0) * Sh::DB + half * DV;
#pragma unroll 1
      for (int c = 0; c < DV; c += 32) {
        float o[32];
        tmem_load_row<32>(o_addr + c, o);
        tmem_ld_wait();
        // (a row tile without a key tile in this part has no O)
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = n > 0 ? o[e] * inv : 0.f;
        if (whole && p.o_bf16 != nullptr) {  // (half a step 2^-8 relative: the up-projection's operand, or out)
          uint4 v4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v4[e] = make_uint4(pack_bf16x2(o[8 * e], o[8 * e + 1]), pack_bf16x2(o[8 * e + 2], o[8 * e + 3]),
                               pack_bf16x2(o[8 * e + 4], o[8 * e + 5]), pack_bf16x2(o[8 * e + 6], o[8 * e + 7]));
          exchange4(v4, lane);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (tok4[r] < u.t.ntok) *reinterpret_cast<uint4*>(out + off4[r] + c) = v4[r];
        } else {
          // fp32: 16 columns at a time, 64 bytes of a row together
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint4 v4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v4[e] = make_uint4(__float_as_uint(o[16 * g + 4 * e]), __float_as_uint(o[16 * g + 4 * e + 1]),
                                 __float_as_uint(o[16 * g + 4 * e + 2]), __float_as_uint(o[16 * g + 4 * e + 3]));
            exchange4(v4, lane);
            const int x = c + 16 * g + (lane & 3) * 4;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              if (tok4[r] >= u.t.ntok) continue;
              float* dst = whole ? p.o_f32 + ((size_t)tok_out * p.vh + head0) * Sh::DB + half * DV + off4[r] -
                                       (lane & 3) * 8 + x
                                 : p.part_o + (pat - (lane & 3) + r) * DV + x;
              *reinterpret_cast<uint4*>(dst) = v4[r];
            }
          }
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (n > 0 && lane == 0) mbar_arrive(&ofree[q]);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0) {
      fold_early(p.tags, p.status);
      // a bad length is the cause of the pages it leads to, whichever was seen first
      if (*reinterpret_cast<volatile unsigned*>(p.tags.words + kTagSeqLen) == p.tags.tag)
        atomicCAS(p.status, kErrPageOob, kErrSeqLen);
      // a replayed graph comes with the same tag: what this call found must not be there for the next
      for (int k = 0; k < 4; ++k) atomicCAS(p.tags.words + k, p.tags.tag, 0u);
    }
    if (*abort_flag) set_status(p.status, kErrTimeout);
    if (*drain_err) force_status(p.status, kErrDrain);
  }
  if (warp == Sh::QK_WARP) {
    tc_fence_after();
    tmem_dealloc(tbase, Sh::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------------------
// Merge of the units that the stretches cut (and zeros for tokens that see no key)
// ---------------------------------------------------------------------------------------
struct MergeParams {
  RowPlan plan;
  int causal, key_tile, halves, chunks, heads_tile, tok_tile, heads_block, vh, db, dv, rows;
  const float* part_o;
  const float* part_lse;
  __nv_bfloat16* o_bf16;   // [tokens][vh][db], or null
  float* o_f32;            // the same when o_bf16 is null
  float* lse;              // natural log, or null
};

// Grid (CTAs of the attention kernel, row slices). Block (c, s) looks after the unit that CTA c goes on
// with, if CTA c - 1 began it: the unit's parts (CTAs c - 1, c, ... in that order) are merged by
// log-sum-exp. A warp takes a row, a lane dv / 32 features. Bound by latency: a few hundred rows a
// block column, two loads deep.
__global__ void __launch_bounds__(256) mlra_rows_merge_kernel(const MergeParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int warp = warp_id(), lane = lane_id(), nwarp = blockDim.x >> 5;
  const int slice = blockIdx.y * nwarp + warp, slices = gridDim.y * nwarp;
  // (a latent result to bf16, half a step 2^-8 relative, for the up-projection's MMAs)
  auto put = [&](size_t at, float v) {
    if (p.o_bf16 != nullptr) p.o_bf16[at] = __float2bfloat16_rn(v);
    else p.o_f32[at] = v;
  };
  if (__ldg(p.plan.hdr + 3) > 0) {
    // token tiles without a key: zeros
    const int tiles = __ldg(p.plan.hdr);
    for (int i = blockIdx.x; i < tiles; i += gridDim.x) {
      const TokenTile t = p.plan.tile[i];
      if (key_tiles(t, p.causal, p.key_tile) > 0) continue;
      for (long long r = slice; r < (long long)t.ntok * p.vh; r += slices) {
        const size_t at = (size_t)t.tok0 * p.vh + r;
        for (int f = lane; f < p.db; f += 32) put(at * p.db + f, 0.f);
        if (lane == 0 && p.lse != nullptr) p.lse[at] = -INFINITY;
      }
    }
  }
  const int c = blockIdx.x;
  const int4 cut = __ldg(p.plan.cut + 2 * c), tk = __ldg(p.plan.cut + 2 * c + 1);
  const int c0 = cut.x, c1 = cut.y, ntok = tk.y;
  if (c == 0 || c0 != c - 1) return;
  const int sub = cut.z / p.halves, half = cut.z % p.halves;
  const int per = p.dv / 32;
  for (int r = slice; r < p.rows; r += slices) {
    const int q = r >> 7, row = r & 127;
    const int tl = row / p.heads_tile, hr = row - tl * p.heads_tile;
    const int tok = q * p.tok_tile + tl;
    if (tl >= p.tok_tile || tok >= ntok) continue;
    float mx = -INFINITY, sum = 0.f;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = 0.f;
    for (int x0 = c0; x0 <= c1; x0 += 4) {
      // four parts' loads under way
      float lv[4], v[4][8];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int x = x0 + g;
        const size_t at = (size_t)(2 * x + (x == c0 ? 1 : 0)) * p.rows + r;
        lv[g] = x <= c1 ? __ldg(p.part_lse + at) : -INFINITY;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[g][e] = x <= c1 && e < per ? __ldg(p.part_o + at * p.dv + e * 32 + lane) : 0.f;
      }
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        if (lv[g] == -INFINITY) continue;
        const float mn = fmaxf(mx, lv[g]);
        const float a = fast_exp2(mx - mn), w = fast_exp2(lv[g] - mn);
        sum = sum * a + w;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = acc[e] * a + w * v[g][e];
        mx = mn;
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int head = (sub / p.chunks) * p.heads_block + (sub % p.chunks) * p.heads_tile + hr;
    const size_t at = (size_t)(tk.x + tok) * p.vh + head;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < per) put(at * p.db + half * p.dv + e * 32 + lane, acc[e] * inv);
    if (lane == 0 && half == 0 && p.lse != nullptr)
      p.lse[at] = sum == 0.f ? -INFINITY : (mx + __log2f(sum)) * kLn2;
  }
}

// ---------------------------------------------------------------------------------------
// Up-projection of many tokens: out[t][h] = out_scale * W^UV_h o~[t][h]
// ---------------------------------------------------------------------------------------
// A persistent grid over (head, tile of 128 tokens) in head-major order, each CTA a contiguous run, so
// a CTA keeps one head's weight in shared memory for most of its run. M = 128 tokens, N = d_h,
// K = SUMK * d_b (summed blocks: the blocks' latents and weights stacked along K); A tiles of 64
// columns come through a ring, two accumulators alternate. Bound by memory: it reads o~ and writes
// out once, 512 bytes for 2 * 128 * 128 FLOPs.
constexpr float kMaxBf16 = 3.3895314e38f;  // the largest bf16 value

template <int DBB_, int DH_, int SUMK_, int STAGES_ = 4, bool STAGED_ = false>
struct UpShape {
  static constexpr int DBB = DBB_, DH = DH_, SUMK = SUMK_, K = DBB * SUMK;
  static constexpr int CW = DBB < 64 ? DBB : 64, ROWB = CW * 2, NKC = K / CW;
  static constexpr int AW = DH < 64 ? DH : 64, WROWB = AW * 2, NATOM = DH / AW;
  static constexpr int ATOM = K * WROWB;
  static constexpr int W_BYTES = NATOM * ATOM;
  static constexpr int A_REG = 128 * ROWB;
  static constexpr int STAGES = STAGES_;
  static constexpr bool STAGED = STAGED_;  // results leave through shared memory (TMA stores)
  static constexpr int OUT_BYTES = STAGED ? 2 * 128 * 128 : 0;  // two halves of 64 columns
  static constexpr int WBOX = DBB < 256 ? DBB : 256;  // rows of the weight map's box
  static constexpr int TMEM_COLS = 2 * DH < 32 ? 32 : 2 * DH;
  static constexpr int OFF_RING = W_BYTES;
  static constexpr int OFF_OUT = OFF_RING + STAGES * A_REG;
  static constexpr int OFF_BAR = OFF_OUT + OUT_BYTES;
  static constexpr int SMEM = OFF_BAR + (2 * STAGES + 2 + 4 + 1) * 8 + 64 + 1024;
  // loads, MMAs, and two groups of four warps that each take half of the result's columns (with one
  // group the expansion of 24,800 tokens took 533 us, bound by its latency)
  static constexpr int THREADS = 320;
  static_assert(W_BYTES % 1024 == 0 && A_REG % 1024 == 0 && SMEM <= 227 * 1024, "layout");
};

// EXPAND: the same product over cached rows instead, for the per-head form: each head's keys c_j W^UK_h
// and values c_j W^UV_h of every cached token, [head][row][K | V], row = b * seq_rows + token (seq_rows:
// the table row's pages, rounded up to whole 128-token tiles, all of which are written); a weight is
// then one of a head's two. Reads the rows once a weight (from L2 after the first), writes 512 bytes
// a token and head: TMA stores of staged tiles, because 64-byte pieces from registers cost more in
// lane exchanges than the product (24,800 tokens of 128 heads: 535 us). The blocks also copy the RoPE
// columns to rows of their own.
// Keys and values are rounded to bf16 (half a step 2^-8 relative), the attention's operands.
// Values are stored finite, infinities and NaN as the largest bf16 values: a masked key's P = 0 then
// adds nothing. A token that does see a cached row with NaN or infinities gets NaN through the
// row's keys, which keep them.
struct UpParams {
  const int* used;       // tokens in use (rows past them are left as they were)
  void* out;             // [tokens][heads][DH]
  int out_f32, heads, total;  // total: tokens of the call
  float out_scale;
  int* status;
  unsigned long long wait_limit_ns;
  // EXPAND
  EarlyTags tags;
  const int* lens;
  const int* page_table;
  int pt_stride, batch, num_pages, heads_block, seq_rows, kv_rows, width, d_c, d_r;
  const __nv_bfloat16* pool;
  __nv_bfloat16* kr;     // [kv_rows][d_r]
};

template <class Sh, bool EXPAND = false>
__global__ void __launch_bounds__(Sh::THREADS)
    mlra_rows_up_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_w2,
                        const __grid_constant__ CUtensorMap map_o, const __grid_constant__ CUtensorMap map_kv,
                        const UpParams p) {
  static_assert(EXPAND == Sh::STAGED && (!EXPAND || Sh::DH == 128), "the expansion's results are staged");
  constexpr int DH = Sh::DH, STAGES = Sh::STAGES, NKC = Sh::NKC;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* wbuf = smem;
  uint8_t* ring = smem + Sh::OFF_RING;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Sh::OFF_BAR);
  uint64_t* empty = full + STAGES;
  uint64_t* wfull = empty + STAGES;
  uint64_t* wfree = wfull + 1;
  uint64_t* dfull = wfree + 1;   // [2]
  uint64_t* dfree = dfull + 2;   // [2]
  uint64_t* drained = dfree + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* drain_err = abort_flag + 1;
  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(wfull, 1);
    mbar_init(wfree, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&dfull[i], 1);
      mbar_init(&dfree[i], 8);
    }
    mbar_init(drained, 1);
    *abort_flag = 0;
    *drain_err = 0;
    fence_mbar_init();
  }
  const int seq_tiles = EXPAND ? (p.pt_stride + 1) / 2 : 1;  // token tiles of a sequence's table row
  const int tiles = EXPAND ? p.batch * seq_tiles : (p.total + 127) / 128;
  const int items = tiles * p.heads * (EXPAND ? 2 : 1);  // (the host keeps this within 32 bits)
  const int per = (items + gridDim.x - 1) / gridDim.x;
  const int lo = (int)min((long long)per * blockIdx.x, (long long)items), hi = min(lo + per, items);
  // item = head * tiles + tile, followed step by step: divisions for both of an item's numbers were most
  // of a role's time (EXPAND's skip still divides by seq_tiles, once an item and role)
  const int h_lo = tiles > 0 ? lo / tiles : 0, tile_lo = lo - h_lo * tiles;
  auto step = [&](int& h, int& tile) {
    if (++tile == tiles) {
      tile = 0;
      ++h;
    }
  };
  auto load_weight = [&](int h) {
    const uint64_t keep = l2_policy_evict_last();
    mbar_arrive_expect_tx(wfull, Sh::W_BYTES);
    for (int a = 0; a < Sh::NATOM; ++a)
      for (int j = 0; j < Sh::SUMK; ++j)
        for (int r = 0; r < Sh::DBB; r += Sh::WBOX)
          tma_load_2d(wbuf + a * Sh::ATOM + (j * Sh::DBB + r) * Sh::WROWB, EXPAND && (h & 1) ? &map_w2 : &map_w, wfull,
                      a * Sh::AW, (EXPAND ? h / 2 : j * p.heads + h) * Sh::DBB + r, keep);
  };
  // the first head's weight does not depend on the kernel before
  if (!EXPAND && threadIdx.x == 0 && lo < hi) load_weight(h_lo);
  grid_dependency_wait();
  if (warp == 1) {
    tmem_alloc(tmem_slot, Sh::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  grid_launch_dependents();

  if (EXPAND && blockIdx.x == 0 && threadIdx.x == 0) clear_status_and_tags(p.status, p.tags);
  const int used = EXPAND ? 0 : __ldg(p.used);
  auto length = [&](int b) { return min(max(__ldg(p.lens + b), 0), p.pt_stride * kPage); };
  // EXPAND: whether the tile lies past its sequence's end
  auto skip = [&](int tile) {
    return EXPAND && (tile % seq_tiles) * 128 >= length(tile / seq_tiles);
  };

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = l2_policy_evict_first(), keep = l2_policy_evict_last();
      uint32_t c = 0, wc = 0, issued = 0, parity = 0;
      int w_parity = -1, head = -1;
      if (!EXPAND && lo < hi) {
        head = h_lo;
        w_parity = 0;
        wc = 1;
      }
      bool ok = true;
      int h = h_lo, tile = tile_lo;
      for (int it = lo; it < hi && ok; ++it, step(h, tile)) {
        const int tok = tile * 128;
        if (skip(tile)) continue;
        int id0 = 0, id1 = 0;  // EXPAND: the tile's two pages (the second may not exist)
        if (EXPAND) {
          const int b = tile / seq_tiles, pg = (tile % seq_tiles) * 2;
          const int* row = p.page_table + (size_t)b * p.pt_stride;
          id0 = __ldg(row + pg);
          id1 = (pg + 1) * kPage < length(b) ? __ldg(row + pg + 1) : id0;
          if (id0 < 0 || id0 >= p.num_pages || id1 < 0 || id1 >= p.num_pages) {
            report_early(p.tags, kTagPageOob);
            id0 = id0 < 0 || id0 >= p.num_pages ? 0 : id0;
            id1 = id1 < 0 || id1 >= p.num_pages ? 0 : id1;
          }
        }
        if (h != head) {
          head = h;
          ok = mbar_wait(wfree, (wc & 1) ^ 1, abort_flag, p.wait_limit_ns);
          if (!ok) break;
          load_weight(h);
          w_parity = wc & 1;
          ++wc;
        }
        for (int kc = 0; kc < NKC && ok; ++kc, ++c) {
          const int s = c % STAGES;
          const uint32_t ph = (c / STAGES) & 1;
          ok = mbar_wait(&empty[s], ph ^ 1, abort_flag, p.wait_limit_ns);
          if (!ok) break;
          mbar_arrive_expect_tx(&full[s], Sh::A_REG);
          issued |= 1u << s;
          parity = (parity & ~(1u << s)) | (ph << s);
          const int f = kc * Sh::CW;
          if (EXPAND) {
            const int x = (h / 2 / p.heads_block) * Sh::DBB + f;
            tma_load_2d(ring + s * Sh::A_REG, &map_o, &full[s], x, id0 * kPage, keep);
            tma_load_2d(ring + s * Sh::A_REG + kPage * Sh::ROWB, &map_o, &full[s], x, id1 * kPage, keep);
            continue;
          }
          tma_load_3d(ring + s * Sh::A_REG, &map_o, &full[s], f % Sh::DBB, (f / Sh::DBB) * p.heads + h, tok, pol);
        }
      }
      for (int s = 0; s < STAGES; ++s)
        if ((issued >> s) & 1)
          if (!mbar_wait_drain(&full[s], (parity >> s) & 1, p.wait_limit_ns)) *drain_err = 1;
      if (w_parity >= 0 && !mbar_wait_drain(wfull, w_parity, p.wait_limit_ns)) *drain_err = 1;
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, DH, false, true);
      const uint32_t w0 = smem_u32(wbuf), a0 = smem_u32(ring);
      uint32_t c = 0, wc = 0, n = 0;
      int head = -1;
      bool ok = true;
      int h = h_lo, tile = tile_lo;
      for (int it = lo; it < hi && ok; ++it, step(h, tile)) {
        if (skip(tile)) continue;
        if (h != head) {
          // the last head's MMAs free its weight
          if (head >= 0) umma_commit(wfree);
          head = h;
          ok = mbar_wait(wfull, wc & 1, abort_flag, p.wait_limit_ns);
          if (!ok) break;
          ++wc;
        }
        const uint32_t d = tbase + (n & 1) * DH;
        ok = mbar_wait(&dfree[n & 1], ((n >> 1) & 1) ^ 1, abort_flag, p.wait_limit_ns);
        for (int kc = 0; kc < NKC && ok; ++kc, ++c) {
          const int s = c % STAGES;
          ok = mbar_wait(&full[s], (c / STAGES) & 1, abort_flag, p.wait_limit_ns);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < Sh::ROWB / 32; ++ks)
            umma_bf16(d, smem_desc(a0 + s * Sh::A_REG + ks * 32, 16, 8 * Sh::ROWB, swizzle_code(Sh::ROWB)),
                      smem_desc(w0 + (kc * Sh::CW + ks * 16) * Sh::WROWB, Sh::ATOM, 8 * Sh::WROWB,
                                swizzle_code(Sh::WROWB)),
                      idesc, (kc > 0 || ks > 0) ? 1u : 0u);
          umma_commit(&empty[s]);
        }
        if (!ok) break;
        umma_commit(&dfull[n & 1]);
        ++n;
      }
      umma_commit(drained);
      if (!mbar_wait_drain(drained, 0, p.wait_limit_ns)) *drain_err = 1;
    }
    __syncwarp();
  } else {
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    uint32_t n = 0;
    if constexpr (EXPAND) {
      // RoPE columns of the pages, 16 bytes a thread
      const int cpr = p.d_r / 8, tid = threadIdx.x - 64;  // 256 threads
      for (int pg = blockIdx.x; pg < p.batch * p.pt_stride; pg += gridDim.x) {
        const int b = pg / p.pt_stride;
        if ((pg - b * p.pt_stride) * kPage >= length(b)) continue;
        int id = __ldg(p.page_table + pg);
        if (id < 0 || id >= p.num_pages) id = 0;  // (reported by the loads)
        for (int i = tid; i < kPage * cpr; i += Sh::THREADS - 64) {
          const int r = i / cpr, x = (i % cpr) * 8;
          const size_t at = (size_t)b * p.seq_rows + (pg - b * p.pt_stride) * kPage + r;
          *reinterpret_cast<uint4*>(p.kr + at * p.d_r + x) = __ldg(
              reinterpret_cast<const uint4*>(p.pool + ((size_t)id * kPage + r) * p.width + p.d_c + x));
        }
      }
    }
    int h = h_lo, tile = tile_lo;
    for (int it = lo; it < hi; ++it, step(h, tile)) {
      const int tok = tile * 128 + row;
      if (skip(tile)) continue;
      const bool ok = __all_sync(0xffffffffu, mbar_wait(&dfull[n & 1], (n >> 1) & 1, abort_flag, p.wait_limit_ns));
      if (!EXPAND && !ok) break;
      tc_fence_after();
      if constexpr (EXPAND) {
        // this group's 64 columns: rows of 128 bytes in the swizzled layout of the store's box, once the
        // last store has read the place
        const int g = (warp - 2) >> 2;
        uint8_t* half = smem + Sh::OFF_OUT + g * (128 * 128);
        const bool storer = ((warp - 2) & 3) == 0 && lane == 0;
        if (storer) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
        __syncwarp();
        if (named_bar_or(1 + g, 128, !ok)) break;  // (a failed wait: the group leaves together)
#pragma unroll
        for (int ci = 0; ci < 64; ci += 32) {
          float v[32];
          tmem_load_row<32>(tbase + lane_base + (n & 1) * DH + 64 * g + ci, v);
          tmem_ld_wait();
          uint4 v4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v4[e] = make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                               pack_bf16x2(v[8 * e + 4], v[8 * e + 5]), pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
          if (h & 1) {  // max and min pass a NaN over
            const __nv_bfloat162 top = __floats2bfloat162_rn(kMaxBf16, kMaxBf16), low = __hneg2(top);
            __nv_bfloat162* h2 = reinterpret_cast<__nv_bfloat162*>(v4);
#pragma unroll
            for (int e = 0; e < 16; ++e) h2[e] = __hmin2(__hmax2(h2[e], low), top);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e)
            *reinterpret_cast<uint4*>(half + swizzle(row * 128 + ci * 2 + e * 16, 128)) = v4[e];
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&dfree[n & 1]);
        fence_proxy_async_smem();
        named_bar_sync(1 + g, 128);
        if (storer) {
          const int y = (h / 2) * p.kv_rows + (tile / seq_tiles) * p.seq_rows + (tile % seq_tiles) * 128;
          asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                           reinterpret_cast<uint64_t>(&map_kv)),
                       "r"((h & 1) * DH + 64 * g), "r"(y), "r"(smem_u32(half))
                       : "memory");
          asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
        ++n;
        continue;
      }
      const int c0 = ((warp - 2) >> 2) * (DH / 2 < 32 ? 32 : DH / 2);
#pragma unroll
      for (int ci = 0; ci < (DH / 2 < 32 ? 32 : DH / 2); ci += 32) {
        const int c = c0 + ci;
        if (c >= DH) break;
        float v[32];
        tmem_load_row<32>(tbase + lane_base + (n & 1) * DH + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] *= p.out_scale;
        if (p.out_f32) {
          // (rows behind the last sequence, tok >= used, stay as they were)
          float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + ((size_t)tok * p.heads + h) * DH + c);
          if (tok < used) {
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
          }
        } else {
          uint4 v4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v4[e] = make_uint4(pack_bf16x2(v[8 * e], v[8 * e + 1]), pack_bf16x2(v[8 * e + 2], v[8 * e + 3]),
                               pack_bf16x2(v[8 * e + 4], v[8 * e + 5]), pack_bf16x2(v[8 * e + 6], v[8 * e + 7]));
          exchange4(v4, lane);
          const int t0 = tok - (lane & 3);
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + ((size_t)t0 * p.heads + h) * DH + c + (lane & 3) * 8;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (t0 + r < used) *reinterpret_cast<uint4*>(dst + (size_t)r * p.heads * DH) = v4[r];
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&dfree[n & 1]);
      ++n;
    }
    // stores still under way read shared memory, and later kernels read what they write
    if (EXPAND && ((warp - 2) & 3) == 0 && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0) {
    if (EXPAND) {  // the call's first kernel: block 0 may not have cleared the status word yet
      if (*abort_flag) report_early(p.tags, kTagTimeout);
      if (*drain_err) report_early(p.tags, kTagDrain);
    } else {
      if (*abort_flag) set_status(p.status, kErrTimeout);
      if (*drain_err) force_status(p.status, kErrDrain);
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tbase, Sh::TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------------------
// E4M3 cache: the sequences' pages as bf16 pages
// ---------------------------------------------------------------------------------------
// One block a page: page i of sequence b becomes page b * pt_stride + i of `dst`. Every E4M3 value is a
// bf16 value, so nothing is rounded; the cache's scales are applied to the query and the result.
// Reads 576 and writes 1152 bytes a token at d_c = 512, once a call, against 640 * heads FLOPs a
// query token and cached token.
__global__ void __launch_bounds__(256) mlra_widen_pages_kernel(const uint8_t* __restrict__ pool, int num_pages,
                                                               const int* __restrict__ page_table, int pt_stride,
                                                               const int* __restrict__ lens, int width,
                                                               __nv_bfloat16* __restrict__ dst, int* status) {
  grid_dependency_wait();  // the buffer may be in use by the work before, and the status word is cleared there
  grid_launch_dependents();
  const int b = blockIdx.y, i = blockIdx.x;
  int n = __ldg(lens + b);
  n = n < 0 ? 0 : n > pt_stride * kPage ? pt_stride * kPage : n;
  if (i * kPage >= n) return;
  int id = __ldg(page_table + (size_t)b * pt_stride + i);
  if (id < 0 || id >= num_pages) {
    if (threadIdx.x == 0) set_status(status, kErrPageOob);
    id = 0;
  }
  const uint4* src = reinterpret_cast<const uint4*>(pool + (size_t)id * kPage * width);
  uint4* out = reinterpret_cast<uint4*>(dst + ((size_t)b * pt_stride + i) * kPage * width);
  for (int x = threadIdx.x; x < kPage * width / 16; x += blockDim.x) {
    const uint4 v = __ldg(src + x);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t o[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t h2 = f16x2_from_e4m3x2(static_cast<uint16_t>(w[e / 2] >> (16 * (e & 1))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
      o[e] = pack_bf16x2(f.x, f.y);
    }
    out[2 * x] = make_uint4(o[0], o[1], o[2], o[3]);
    out[2 * x + 1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

}  // namespace mlra
