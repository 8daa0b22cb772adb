// Tile GEMM of two MXFP4 operands (both E2M1 with a UE8M0 scale per 32 along
// K) for the dense layer and for the experts' products on sorted rows.
//
// On gfx950 the scaled MFMA multiplies 4-bit by 4-bit operands in half the
// cycles of 8-bit ones, with half the operand bytes, so a 128-K step of a 256
// x 256 tile is 64 MFMAs of 16 cycles per wave against 32 KiB of operands.
// Large tiles are bound by the issue of MFMAs among LDS reads and copies, and by
// the clock that the chip's power leaves: 8192 x 28672 x 8192 takes 790 us (4.9
// PFLOP/s; 830 to 870 called back to back), the matrix cores busy 0.62 of the
// cycles at 1.9 GHz.  MFMAs alone would take 588 at 1.6 GHz, with the copies 652,
// with the LDS reads 686: the clock rises with the idle cycles and makes up for a
// part of them (a loop of MFMAs on registers: 7.5 PFLOP/s on random codes, 9.0 on
// zeros).  The 256 x 256 tiles use all 512 registers and four spilled ones, read
// back once a tile.  The experts' tiles are bound by their start and end, which
// nothing covers: 4096 tokens,
// 128 experts, k 8, 1536 x 2048 102 us (3.2 TB/s of the 331 MB that they cannot do
// without); 14 us per 256 x 128 tile, of which the sixteen steps are 7.5, the
// stores 2, staging them 1, the next tile's decoding and sources 1.5.
//
//  * Workgroup tile 32 NA weight rows x 32 NB activation rows, four waves as 2
//    x 2, each 16 NA x 16 NB: NA x NB v_mfma_scale_f32_16x16x128 per 128-K
//    step, the weight as the A operand; lane (i, g) ends with acc[a][b][j] =
//    D[n = wn 16 NA + 16a + 4g + j][m = wm 16 NB + 16b + i].
//  * A step's operands are copied straight into one of four LDS slots
//    (buffer_load ... lds); the slot's fragments are read into registers one step
//    ahead, while the MFMAs of the step before run, and the slot is refilled
//    right after: early in step s the copies of s + 1 have landed, those of s + 2
//    and s + 3 are in flight and those of s + 4 go out between its MFMAs.  One
//    barrier per step.
//  * Where a round of the chip holds all tiles, a workgroup has one, and two
//    groups of four waves: each group runs every other pair of steps on slots of
//    its own, so that a SIMD has a second wave to run while one waits for its
//    reads, and the two add their sums through LDS at the end.  (1000 x 4096 x
//    4096, the GEMM alone: 14.3 us, with one group 15.5; 2048 x 2048 x 8192 23.2
//    and 26.4.  A step takes 0.26 us then: its copies alone 0.18, its MFMAs 0.16,
//    its reads 0.11.)
//  * Persistent beyond that: a workgroup runs tiles b, b + gridDim.x, ...  The
//    copy stream has its own position ("cursor"), four steps ahead, and runs on
//    into the next tiles while a tile ends and is stored.
//  * Scales: the packed operands' scale tiles of a pair of steps (256 K) are
//    1 KiB per 128-row group: one copy per pair.  Of rows by index (kRows) a
//    copy touches one cache line per row, so it brings four steps' bytes of each
//    (per step instead: a quarter slower on 4096 tokens, 128 experts, 1536 x
//    2048).
#include <algorithm>

#include "fp4.hpp"

namespace mxfp8 {

namespace {

using tile::buffer_rsrc;
using tile::i4v;

constexpr int kThreads = 256;   // of a group of waves
constexpr int kRing = 4;        // steps in LDS

// tile::b2l_16 and b2l_4 with the LDS address as a base and a constant: one
// scalar add into m0.
template <int kAt>
__device__ __forceinline__ void b2l_16(uint32_t voff, i4v rsrc, uint32_t soff, uint32_t lds) {
  asm volatile("s_add_u32 m0, %3, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds" ::"v"(voff), "s"(rsrc),
               "s"(soff), "s"(lds), "n"(kAt)
               : "memory", "m0", "scc");
}
template <int kAt>
__device__ __forceinline__ void b2l_4(uint32_t voff, i4v rsrc, uint32_t soff, uint32_t lds) {
  asm volatile("s_add_u32 m0, %3, %4\n\ts_nop 0\n\tbuffer_load_dword %0, %1, %2 offen lds" ::"v"(voff), "s"(rsrc),
               "s"(soff), "s"(lds), "n"(kAt)
               : "memory", "m0", "scc");
}
using tile::lds_addr;

// How the activations come: the packed operand; rows by index from row-major
// quantized ones; or bf16 rows, quantized by the workgroup itself.
constexpr int kPacked = 0, kRows = 1, kFused = 2;

template <int NA, int NB, int kX, int kGroups>
struct Fp4Lds {
  static constexpr int kRowsN = 32 * NA, kRowsM = 32 * NB;
  static constexpr int kW = kRowsN * 64;
  static constexpr int kSlot = kW + (kX == kFused ? 0 : kRowsM * 64);   // one 128-K step
  static constexpr int kRunsW = NA / 4, kRunsX = kX == kPacked ? (NB + 3) / 4 : 0;   // scale runs of 1 KiB per pair
  static constexpr int kScale = (kRunsW + kRunsX) * 1024;  // one pair of steps
  static constexpr int kPitch = 32 * NA;                   // bytes of a staged output row
  // Rows staged at a time: eight where that lets two workgroups share a compute
  // unit's 160 KiB.
  static constexpr int kEpiRows = kX != kPacked && NA == 4 ? 8 : 16;
  static constexpr int kEpiWave = kEpiRows * kPitch;
  static constexpr int kBiasSlot = 512;                    // a tile's bias, 256 bytes per wave column
  static constexpr int kScaleAt = kRing * kSlot;
  static constexpr int kGroup = kScaleAt + kRing / 2 * kScale;   // one wave group's slots and scales
  // Scales of gathered rows: one copy brings 16 bytes (four steps) of 64 / kEntry
  // times a wave's kEntry rows, kChunk steps; two chunks.
  static constexpr int kEntry = 8 * NB, kChunk = 32 / NB;
  static constexpr int kXsAt = kGroups * kGroup;
  static constexpr int kEpiAt = kXsAt + (kX == kRows ? 2 * 4096 : 0);
  static constexpr int kBiasAt = kEpiAt + kGroups * 4 * kEpiWave;
  static constexpr int kIndexAt = kBiasAt;                 // kRows: row indices instead of a bias
  static constexpr int kJobAt = kBiasAt + (kX == kRows ? 1024 : kRing * kBiasSlot);
  static constexpr int kBytes = kJobAt + 8 * 32;           // (the cursor is at most five tiles ahead)
  static_assert(kBytes <= 160 * 1024, "LDS of a compute unit");
  // kFused, behind all that: per step the tile's rows and their scale bytes.
  static constexpr int kFusedStep = kX == kFused ? kRowsM * 64 + kRowsM * 4 : 0;
  static constexpr int kCopies = NA / 2 + (kX == kFused ? 0 : NB / 2);   // per wave and step, without scales
};

struct Fp4Args {
  const uint8_t* q;        // activations: packed, or row-major [x_rows, K / 2]
  const uint8_t* s;        // their scales; row-major rows are s_pitch bytes apart
  uint32_t q_bytes, s_bytes, s_pitch;   // kRows: sizes of q and s
  const uint16_t* x;       // kFused: bf16 [x_rows, K], row stride ldx
  int64_t ldx;
  int x_rows;
  int M, K;                // dense: activation rows
  const uint8_t* wp;
  const uint8_t* wsp;
  int N;
  const uint16_t* bias;
  uint16_t* y;
  int64_t ldy;
  int past;                // y is stored around the caches
  // experts
  int R, E, topk;
  const int* slots;        // or null: row r of q
  const int* offsets;
};

// One tile of the list.
struct Fp4Job {
  int row0, row_end;       // output rows [row0, row_end) at most
  int col0;
  int wgroup;              // its first 128-row group of the packed weight
  int live;
};

// Tiles of the dense layer: groups of kGroupM M-tiles, N inside, so that the
// workgroups of a die share operands in its L2.
constexpr int kGroupM = 4;
template <int NA, int NB>
struct DenseTiles {
  int tiles_m, tiles_n, total;
  __device__ DenseTiles(const Fp4Args& p) {
    tiles_m = (p.M + 32 * NB - 1) / (32 * NB);
    tiles_n = (p.N + 32 * NA - 1) / (32 * NA);
    total = tiles_m * tiles_n;
  }
  __device__ Fp4Job job(const Fp4Args& p, int b) const {
    Fp4Job j;
    j.live = b < total;
    const int logical = xcd_remap(j.live ? b : 0, total);
    const int per_group = kGroupM * tiles_n;
    const int group = logical / per_group, first_m = group * kGroupM;
    const int gm = min(tiles_m - first_m, kGroupM);
    const int in_group = logical - group * per_group;
    const int tm = first_m + in_group % gm, tn = in_group / gm;
    j.row0 = tm * 32 * NB;
    j.row_end = p.M;
    j.col0 = tn * 32 * NA;
    j.wgroup = j.col0 / kGroupRows;
    return j;
  }
};

// Tiles of the experts: expert by expert, weight tile by weight tile, the
// expert's row tiles inside.  Lane l holds experts 4 l .. 4 l + 3.
template <int NA, int NB>
struct ExpertTiles {
  int first[4], rows[4], start[4];
  int tiles_n, total, kept;
  __device__ ExpertTiles(const Fp4Args& p) {
    const int lane = threadIdx.x & 63;
    tiles_n = (p.N + 32 * NA - 1) / (32 * NA);
    int sum = 0, n[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = 4 * lane + u;
      first[u] = min(max(p.offsets[min(e, p.E)], 0), p.R);
      rows[u] = max(min(p.offsets[min(e + 1, p.E)], p.R) - first[u], 0);
      n[u] = (rows[u] + 32 * NB - 1) / (32 * NB) * tiles_n;
      sum += n[u];
    }
    int run = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int o = __shfl_up(run, off);
      if (lane >= off) run += o;
    }
    total = __builtin_amdgcn_readlane(run, 63);
    run -= sum;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      start[u] = run;
      run += n[u];
    }
    kept = max(__builtin_amdgcn_readfirstlane(p.offsets[p.E]), 0);
  }
  __device__ Fp4Job job(const Fp4Args& p, int b) const {
    Fp4Job j;
    j.live = b < total;
    if (!j.live) {
      j.row0 = j.row_end = j.col0 = 0;
      j.wgroup = 0;
      return j;
    }
    const int t = xcd_remap(b, total);
    // The last expert that starts at or before t (one without tiles starts
    // where the next one does).
    int at = -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) at += __popcll(__ballot(start[u] <= t));
    const int e = __builtin_amdgcn_readfirstlane(at);
    const int l = e >> 2, u = e & 3;
    auto pick = [&](const int (&v)[4]) {
      return __builtin_amdgcn_readlane(u == 0 ? v[0] : u == 1 ? v[1] : u == 2 ? v[2] : v[3], l);
    };
    const int n = pick(rows), r0 = pick(first), inside = t - pick(start);
    const int tiles_m = (n + 32 * NB - 1) / (32 * NB);
    const int tn = inside / tiles_m, tm = inside - tn * tiles_m;
    j.row0 = r0 + tm * 32 * NB;
    j.row_end = r0 + n;
    j.col0 = tn * 32 * NA;
    j.wgroup = e * ((p.N + kGroupRows - 1) / kGroupRows) + j.col0 / kGroupRows;
    return j;
  }
};

}  // namespace

template <int NA, int NB, int kX, bool kExperts, int kGroups>
__global__ __launch_bounds__(kThreads * kGroups, (kGroups == 2 || Fp4Lds<NA, NB, kX, kGroups>::kBytes > 80 * 1024
                                                      ? 1 : 2)) void gemm_fp4_kernel(Fp4Args p) {
  using L = Fp4Lds<NA, NB, kX, kGroups>;
  constexpr bool kOwnScales = kX != kPacked;   // a lane's scale in a byte of its own
  using Tiles = typename std::conditional<kExperts, ExpertTiles<NA, NB>, DenseTiles<NA, NB>>::type;
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];

  const int tid = threadIdx.x, lane = tid & 63;
  const int group = kGroups == 1 ? 0 : __builtin_amdgcn_readfirstlane(tid >> 8);
  const int wave = __builtin_amdgcn_readfirstlane((tid >> 6) & 3);   // in its group
  const int wn = wave >> 1, wm = wave & 1;
  const int li = lane & 15, lg = lane >> 4;
  const int KS4 = p.K / 128;                                  // 128-K steps: even, at least 2
  const int GN = (p.N + kGroupRows - 1) / kGroupRows;         // weight groups (of one expert)
  const int GM = kX != kPacked ? 0 : (p.M + kGroupRows - 1) / kGroupRows;
  const uint32_t gbytes = (uint32_t)KS4 * kTileBytes, sbytes = (uint32_t)KS4 * 2 * kTileScaleBytes;
  const Tiles tiles(p);

  if constexpr (kExperts) zero_rows(p.y, p.ldy, tiles.kept, p.R, p.N, kGroups * kThreads / 64);
  if ((int)blockIdx.x >= tiles.total) return;

  // ------------------------------------------------------------ the copies
  // The cursor: step cq of this workgroup's tile ctile; sources of its tile.  Past the last
  // tile the sources are empty: the copies bring zeros, without touching
  // memory, and every wait counts the same.
  int cq = 2 * group, ctile = 0;
  i4v w0, w1, x0, x1, sc, xsr;
  uint32_t vx[NB / 2], vxhi = 0, vxs = 0;
  uint8_t* const ring = smem + group * L::kGroup;
  const uint32_t lds0 = lds_addr(ring) + (uint32_t)wave * 1024u;   // this wave's share of a region
  const uint32_t lo16 = (uint32_t)lane * 16u;
  const uint32_t band = (uint32_t)KS4 * kPieceBytes;          // bytes of a 16-row band
  auto bias_slot = [&](int t) { return smem + L::kBiasAt + (t & (kRing - 1)) * L::kBiasSlot; };
  uint8_t* const index_slot = smem + L::kIndexAt + wave * 256;
  // Decoding a tile takes a wave some hundred instructions, so each is decoded
  // once, a tile before the cursor gets to it, and kept in LDS (every wave
  // writes the same values and reads its own).
  auto job_slot = [&](int t) { return reinterpret_cast<int4*>(smem + L::kJobAt + (t & 7) * 32); };
  auto put_job = [&](int t) {
    const Fp4Job j = tiles.job(p, (int)blockIdx.x + t * (int)gridDim.x);
    job_slot(t)[0] = make_int4(j.row0, j.row_end, j.col0, j.wgroup);
    job_slot(t)[1].x = j.live;
    return j;
  };
  auto get_job = [&](int t) {
    const int4 v = job_slot(t)[0];
    Fp4Job j;
    j.row0 = __builtin_amdgcn_readfirstlane(v.x);
    j.row_end = __builtin_amdgcn_readfirstlane(v.y);
    j.col0 = __builtin_amdgcn_readfirstlane(v.z);
    j.wgroup = __builtin_amdgcn_readfirstlane(v.w);
    j.live = __builtin_amdgcn_readfirstlane(job_slot(t)[1].x);
    return j;
  };
  // The row of the tile that entry `lane` of the wave's share stands for:
  // rows 16 wave + 64 i + (0 .. 15), i = lane / 16.
  const int my_row = 64 * (lane >> 4) + 16 * wave + (lane & 15);
  auto fetch_index = [&](const Fp4Job& j) {
    if constexpr (kX == kRows) {
      if (p.slots != nullptr) {
        const i4v r = buffer_rsrc(p.slots, j.live ? (uint32_t)p.R * 4u : 0u);
        b2l_4<0>((uint32_t)min(j.row0 + my_row, j.row_end - 1) * 4u, r, 0u, lds_addr(index_slot));
      }
    }
  };
  auto set_sources = [&](const Fp4Job& j, int t) {
    const int last = GN - 1 - j.col0 / kGroupRows;            // groups behind the first one
    const uint32_t live = j.live ? 1u : 0u;
    w0 = buffer_rsrc(p.wp + (size_t)j.wgroup * gbytes, live * gbytes);
    if constexpr (NA == 8) w1 = buffer_rsrc(p.wp + (size_t)(j.wgroup + min(1, last)) * gbytes, live * gbytes);
    const uint8_t* srun = p.wsp + (size_t)j.wgroup * sbytes;  // this wave's scale run
    if (NA == 8 && wave == 1) srun = p.wsp + (size_t)(j.wgroup + min(1, last)) * sbytes;
    if constexpr (kX == kRows) {
      int row = min(j.row0 + my_row, j.row_end - 1);
      if (p.slots != nullptr) {
        row = *reinterpret_cast<const int*>(index_slot + lane * 4);
        row = j.live ? row / p.topk : 0;
      }
      row = j.live ? row : 0;
      xsr = buffer_rsrc(p.s, live * p.s_bytes);
      x0 = buffer_rsrc(p.q, live * p.q_bytes);
      vxs = (uint32_t)__shfl(row, lane % L::kEntry) * p.s_pitch + (uint32_t)(lane / L::kEntry) * 16u;
#pragma unroll
      for (int i = 0; i < NB / 2; ++i) {
        const uint32_t r = (uint32_t)__shfl(row, 16 * i + (lane >> 2));
        const int tr = 64 * i + 16 * wave + (lane >> 2);      // its row in the tile
        vx[i] = r * (uint32_t)(p.K / 2) + (uint32_t)((lane & 3) ^ swz(tr)) * 16u;
      }
    } else if constexpr (kX == kPacked) {
      const int xg = j.row0 / kGroupRows;
      x0 = buffer_rsrc(p.q + (size_t)xg * gbytes, live * gbytes);
      if constexpr (NB == 8) x1 = buffer_rsrc(p.q + (size_t)min(xg + 1, GM - 1) * gbytes, live * gbytes);
      const int first = NB == 2 ? (j.row0 % kGroupRows) / 16 : 0;
      vx[0] = (uint32_t)(first + wave) * band + lo16;
      vxhi = vx[0] + 4u * band;
      if (wave >= L::kRunsW) srun = p.s + (size_t)min(xg + wave - L::kRunsW, GM - 1) * sbytes;
    }
    sc = buffer_rsrc(srun, live * sbytes);
    if constexpr (!kExperts) {
      if (p.bias != nullptr && wm == 0 && group == 0) {
        // this wave column's 16 NA bias values, by whole words (an odd N's last
        // word holds one value that is not the bias's and reaches no output)
        const int c = j.col0 + wn * 16 * NA;
        const uint32_t words = (uint32_t)(max(0, min(16 * NA, p.N - c)) + 1) / 2;
        const i4v r = buffer_rsrc(reinterpret_cast<const uint8_t*>(p.bias) + 2 * (size_t)c, live * words * 4u);
        b2l_4<0>((uint32_t)lane * 4u, r, 0u, lds_addr(bias_slot(t) + wn * 256));
      }
    }
  };
  const uint32_t vw = (uint32_t)wave * band + lo16;
  // Copy k of step q of the cursor's tile into the ring slot at st (of this
  // wave's share: + 1024 wave): calls go(LDS offset in the slot, vector offset,
  // source, scalar offset).
  const uint32_t vwhi = vw + 4u * band;
  auto source = [&](auto kCopy, int q, auto&& go) {
    constexpr int k = decltype(kCopy)::value;
    const uint32_t off = (uint32_t)q * kPieceBytes;
    if constexpr (k < NA / 2) {
      go(std::integral_constant<int, k * 4096>{}, k & 1 ? vwhi : vw, k < 2 ? w0 : w1, off);
    } else {
      constexpr int i = k - NA / 2;
      constexpr std::integral_constant<int, L::kW + i * 4096> at;
      if constexpr (kX == kRows) go(at, vx[i], x0, (uint32_t)q * 64u);
      else go(at, i & 1 ? vxhi : vx[0], i < 2 ? x0 : x1, off);
    }
  };
  auto issue = [&](auto kCopy, int q, uint32_t st) {
    source(kCopy, q, [&](auto at, uint32_t v, i4v r, uint32_t off) { b2l_16<decltype(at)::value>(v, r, off, st); });
  };
  const bool has_run = wave < L::kRunsW + L::kRunsX;
  auto issue_scales = [&](int q, int pair) {
    if (has_run)
      b2l_16<L::kScaleAt>(lo16, sc, (uint32_t)q * 2u * kTileScaleBytes, lds0 + (uint32_t)(pair * L::kScale));
  };
  // The scales of the cursor's pair of steps (q the first): a packed operand's
  // run, and at the start of a chunk the gathered rows'.
  int xput = 0;                                               // chunk buffer to fill next
  auto issue_all_scales = [&](int q, int pair) {
    issue_scales(q, pair);
    if constexpr (kX == kRows) {
      if (q % L::kChunk == 0) {
        b2l_16<L::kXsAt>(vxs, xsr, (uint32_t)q * 4u, lds0 + (uint32_t)xput * 4096u);
        xput ^= 1;
      }
    }
  };
  // Sources of tile ctile (its indices are in LDS), and the next one decoded and
  // its indices on their way: into the place of those just read.
  auto advance_tile = [&]() {
    set_sources(get_job(ctile), ctile);
    const Fp4Job next = put_job(ctile + 1);
    if constexpr (kX == kRows) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    fetch_index(next);
  };

  // ------------------------------------------------------------ fragments
  struct Frags {
    i4v a[NA], b[NB];
    int sa[2], sb[kOwnScales ? NB : 2];
  };
  // A wave's rows of a 128-row group start at 16 NA wn (NA = 8: its own group)
  // and share the swizzle of row li.
  const int offA = tile_off(wn * 16 * NA + li, lg);
  const int offB = (kX == kFused ? L::kBytes : L::kW) + tile_off(wm * 16 * NB + li, lg);
  // Scale words of a packed operand: lane (i, g) supplies MX block g of the
  // step, block g % 2 of its scale tile g / 2; word e holds rows 16e + i + 32k
  // in byte k; rows that start at 32 z of the group: the word shifted by 8 z.
  const int offS = (lg >> 1) * kTileScaleBytes + scale_off(li, lg & 1);
  const int shiftA = NA == 8 ? 0 : 16 * wn;
  const int offSA = (NA == 8 ? wn * 1024 : 0) + offS;
  const int offSB = L::kRunsW * 1024 + (NB == 8 ? wm * 1024 : 0) + offS;
  // Gathered rows: [wave][four steps][entry] of 16 scale bytes, row 64 i + 16 w +
  // r at entry 16 i + r of wave w's share, so 16-row block q in wave q % 4's, at
  // entries 16 (q / 4) ..
  const int offXS = li * 16 + lg + (NB == 8 ? wm * 512 : NB == 4 ? wm * 256 : wm * 2048);
  int shiftB = NB == 8 ? 0 : NB == 4 ? 16 * wm : 8 * wm;     // NB == 2: and the tile's half of its group
  constexpr int kReads = 4 + NA + NB + (kOwnScales ? NB - 2 : 0);
  // Read r of a step's fragments: the scales first.
  auto read_part = [&](int r, Frags& f, const uint8_t* st, const uint8_t* sct, const uint8_t* xs) {
    constexpr int kSB = kOwnScales ? NB : 2;
    if (r < 2) {
      f.sa[r] = (int)((uint32_t)*reinterpret_cast<const int*>(sct + offSA + 128 * r) >> shiftA);
    } else if (r < 2 + kSB) {
      const int e = r - 2;
      // xs: kRows block q = NB wm + e; kFused: the step's rows
      if constexpr (kX == kRows) {
        f.sb[e] = xs[offXS + (NB == 8 ? (e & 3) * 1024 + (e >> 2) * 256 : e * 1024)];
      } else if constexpr (kX == kFused) {
        f.sb[e] = xs[L::kBytes + L::kRowsM * 64 + (wm * 16 * NB + 16 * e + li) * 4 + lg];
      } else {
        f.sb[e] = (int)((uint32_t)*reinterpret_cast<const int*>(sct + offSB + 128 * e) >> shiftB);
      }
    } else if (r < 2 + kSB + NA) {
      const int a = r - 2 - kSB;
      f.a[a] = *reinterpret_cast<const i4v*>(st + offA + 1024 * a);
    } else {
      const int bb = r - 2 - kSB - NA;
      f.b[bb] = *reinterpret_cast<const i4v*>((kX == kFused ? xs : st) + offB + 1024 * bb);
    }
  };

  v4f acc[NA][NB];
  // One step: its fragments are in cur; reads those of the step behind it from
  // slot `next` (scales at nsc) and copies step q of the cursor's tile into
  // slot `free`.  The scales of the cursor's pair go out first in a pair's
  // second step (kSecond): until then the pair they replace is still read.
  // The MFMAs go in blocks of four, each with a copy inside where there is one
  // to issue, and the fragment reads spread between them.  The first kHead
  // blocks run before the barrier, over the end of the step's own reads.
  auto step = [&](auto kSecond, const Frags& cur, Frags& nxt, uint32_t free, const uint8_t* next, int pair,
                  const uint8_t* nsc, const uint8_t* xs, int q) {
    constexpr int kBlocks = NA * NB / 4, kHead = kBlocks / 8, kGaps = kBlocks - kHead;
    // (A small tile's few MFMAs only cover the reads if all go out before them.)
    constexpr bool kReadsFirst = kBlocks <= 4;
    tile::static_for<0, kBlocks>([&](auto J) {
      constexpr int j = decltype(J)::value, g = j - kHead;
      constexpr int a = 4 * j % NA, bb = 4 * j / NA;
      if constexpr (g == 0) {
        // Every wave has read this step's fragments (the slot may be refilled),
        // and the next step's copies have landed: the operand copies of the
        // kRing - 2 steps behind it may be in flight; what else was issued since
        // makes the wait only stricter.
        tile::wait_vmcnt<(kRing - 2) * L::kCopies>();
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (decltype(kSecond)::value) issue_all_scales(q - 1, pair);
        if constexpr (kReadsFirst)
          tile::static_for<0, kReads>([&](auto R) { read_part(decltype(R)::value, nxt, next, nsc, xs); });
      }
      // op_sel: the byte of the scale word (packed), byte 0 of the lane's own
      // (gathered).
      constexpr int selA = a >> 1, selB = kOwnScales || NB == 2 ? 0 : bb >> 1, sb = kOwnScales ? bb : bb & 1;
      constexpr int c0 = g < 0 ? 0 : g * L::kCopies / kGaps, c1 = g < 0 ? 0 : (g + 1) * L::kCopies / kGaps;
      if constexpr (c1 > c0) {
        source(std::integral_constant<int, c0>{}, q, [&](auto at, uint32_t v, i4v r, uint32_t off) {
          mfma16x4_fp4<selA, selB, true, decltype(at)::value>(acc[a][bb], acc[a + 1][bb], acc[a + 2][bb], acc[a + 3][bb],
                                                              cur.a + a, cur.b[bb], cur.sa[0], cur.sa[1], cur.sb[sb], v,
                                                              r, off, free);
        });
      } else {
        mfma16x4_fp4<selA, selB, false, 0>(acc[a][bb], acc[a + 1][bb], acc[a + 2][bb], acc[a + 3][bb], cur.a + a,
                                           cur.b[bb], cur.sa[0], cur.sa[1], cur.sb[sb]);
      }
      if constexpr (g >= 0) {
        tile::static_for<c0 + 1, c1>([&](auto C) { issue(C, q, free); });
        if constexpr (!kReadsFirst)
          tile::static_for<g * kReads / kGaps, (g + 1) * kReads / kGaps>(
              [&](auto R) { read_part(decltype(R)::value, nxt, next, nsc, xs); });
      }
      __builtin_amdgcn_sched_barrier(0);
    });
  };
  using T = std::true_type;
  using F = std::false_type;

  // ------------------------------------------------------------ start
  auto slot = [&](int s) { return ring + s * L::kSlot; };
  auto fill = [&](int s) { return lds0 + (uint32_t)(s * L::kSlot); };
  // Scales of gathered rows for step q of a tile, in the chunk buffer in use.
  int xget = 0;
  auto xs_at = [&](int q) -> const uint8_t* {
    if constexpr (kX == kPacked) return nullptr;
    if constexpr (kX == kFused) return smem + (kGroups == 1 ? q : min(q, KS4 - 1)) * L::kFusedStep;
    return smem + L::kXsAt + xget * 4096 + q % L::kChunk / 4 * (L::kEntry * 16) + (q & 3) * 4;
  };
  auto scale_slot = [&](int pair) { return ring + L::kScaleAt + pair * L::kScale; };
  // Moves the cursor over a pair of steps.
  auto stop_copies = [&]() {
    w0[2] = 0;
    if constexpr (kX == kPacked) x0[2] = 0;
    sc[2] = 0;
  };
  auto move_cursor = [&]() {
    cq += 2 * kGroups;
    if constexpr (kGroups == 2) {
      if (cq >= KS4) stop_copies();
    } else if (cq == KS4) {
      cq = 0;
      ++ctile;
      if constexpr (kX == kRows) {
        // The new tile's indices were fetched a tile ago: with fewer steps per
        // tile than slots their copies may not have been waited for.
        if (KS4 < kRing) tile::wait_vmcnt<0>();
      }
      advance_tile();
    }
  };
  fetch_index(put_job(0));
  if constexpr (kX == kRows) tile::wait_vmcnt<0>();
  advance_tile();
  if (kGroups == 2 && cq >= KS4) stop_copies();
  for (int pair = 0; pair < kRing / 2; ++pair) {
    issue_all_scales(cq, pair);
    tile::static_for<0, L::kCopies>([&](auto C) { issue(C, cq, fill(2 * pair)); });
    tile::static_for<0, L::kCopies>([&](auto C) { issue(C, cq + 1, fill(2 * pair + 1)); });
    if (kX == kRows && cq + 2 == KS4) tile::wait_vmcnt<0>();   // (the second tile's indices)
    move_cursor();
  }
  // Step 0 has landed: at most the operand copies behind it are in flight.
  tile::wait_vmcnt<(kRing - 1) * L::kCopies>();
  __builtin_amdgcn_s_barrier();
  Frags f0, f1;
  auto tile_shift = [&](const Fp4Job& j) {
    if constexpr (NB == 2 && kX == kPacked) shiftB = 8 * (2 * ((j.row0 % kGroupRows) / 64) + wm);
  };
  Fp4Job cur = get_job(0);
  tile_shift(cur);
  tile::static_for<0, kReads>([&](auto R) { read_part(decltype(R)::value, f0, slot(0), scale_slot(0), xs_at(2 * group)); });

  // kFused: the tile's rows into LDS, sixteen lanes per row and step, as in the
  // packed quantizer; rows past the last keep what was there (their outputs are
  // not stored).  Bound by each wave's chain of instructions (64 rows of 1024: 3
  // us, with one group of waves 5), not by the loads (all rows' in flight: slower).
  auto quantize_rows = [&](const Fp4Job& j) {
    constexpr int kBatch = 4;
    const int l = tid & 15, n = j.row_end - j.row0;
#pragma unroll
    for (int r0 = 0; r0 < L::kRowsM; r0 += 16 * kGroups) {
      if (r0 >= n) break;
      const int r = r0 + (tid >> 4);
      const bool in = r < n;
      int64_t row = in ? j.row0 + r : j.row0;
      if (kExperts && p.slots != nullptr) row = min((uint32_t)p.slots[row] / (uint32_t)p.topk, (uint32_t)p.x_rows - 1u);
      const uint16_t* xr = p.x + row * p.ldx + l * 8;
      for (int k0 = 0; k0 < KS4; k0 += kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          v[u] = k0 + u < KS4 ? *reinterpret_cast<const uint4*>(xr + (k0 + u) * 128) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
          const uint32_t sb = fp4_scale_byte(quad_max(fp4_absmax8(v[u])));
          const uint32_t code = cvt8_fp4(v[u], fp4_scale_value(sb));
          uint8_t* d = smem + L::kBytes + (k0 + u) * L::kFusedStep;
          if (in && k0 + u < KS4) {
            *reinterpret_cast<uint32_t*>(d + tile_off(r, l >> 2) + (l & 3) * 4) = code;
            if ((l & 3) == 0) d[L::kRowsM * 64 + r * 4 + (l >> 2)] = (uint8_t)sb;
          }
        }
      }
    }
    __syncthreads();
  };

  int pair = 0, t = 0;
  for (;;) {
    if constexpr (kX == kFused) {
      // (every wave's reads of the last tile's rows are done at its last step's
      // barrier, but for those of that step itself)
      if (t > 0) __syncthreads();
      quantize_rows(cur);
      tile::static_for<0, kReads>([&](auto R) {
        constexpr int r = decltype(R)::value;
        if constexpr ((r >= 2 && r < 2 + NB) || r >= 2 + NB + NA) read_part(r, f0, nullptr, nullptr, xs_at(2 * group));
      });
    }
    if (!kExperts && p.bias != nullptr && group == 0) {
      const uint8_t* bs = bias_slot(t) + wn * 256;
#pragma unroll
      for (int a = 0; a < NA; ++a) {
        const uint2 w = *reinterpret_cast<const uint2*>(bs + (16 * a + 4 * lg) * 2);
        const v4f v = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
#pragma unroll
        for (int c = 0; c < NB; ++c) acc[a][c] = v;
      }
    } else {
#pragma unroll
      for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int c = 0; c < NB; ++c) acc[a][c] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
      for (int c = 0; c < NB; ++c) asm volatile("" : "+a"(acc[a][c]));
    const Fp4Job nxt = get_job(t + 1);
    // (an odd number of pairs: the second group's last one is zeros)
    const int KSe = kGroups == 1 ? KS4 : (KS4 + 3) / 4 * 4;
    for (int q = 2 * group; q < KSe; q += 2 * kGroups) {
      const int npair = (pair + 1) & (kRing / 2 - 1);
      step(F{}, f0, f1, fill(2 * pair), slot(2 * pair + 1), pair, scale_slot(pair) + 2 * kTileScaleBytes,
           xs_at(q + 1), cq);
      // (the last step of a tile reads the next tile's first fragments)
      const int qn = kGroups == 2 ? q + 4 : q + 2 == KS4 ? 0 : q + 2;
      if (qn == 0) tile_shift(nxt);
      if (kX == kRows && qn % L::kChunk == 0) xget ^= 1;
      step(T{}, f1, f0, fill(2 * pair + 1), slot(2 * npair), pair, scale_slot(npair), xs_at(qn), cq + 1);
      move_cursor();
      pair = npair;
    }
    // The last MFMAs must retire before the accumulators are read.
    asm volatile("s_nop 15\n\ts_nop 15\n\ts_nop 15" ::: "memory");

    if constexpr (kGroups == 2) {
      // The two groups' sums: each takes half of the columns, k = NB / 2 group ..,
      // and gets the other's part of them through LDS, in the place of the slots.
      tile::wait_vmcnt<0>();
      __syncthreads();
      constexpr int kH = NB / 2;
      static_assert(2 * 4 * NA * kH * 1024 <= 2 * L::kGroup, "the exchanged sums");
      v4f* const out = reinterpret_cast<v4f*>(smem) + ((group * 4 + wave) * NA * kH) * 64 + lane;
      const v4f* const in = reinterpret_cast<const v4f*>(smem) + (((1 - group) * 4 + wave) * NA * kH) * 64 + lane;
#pragma unroll
      for (int k = 0; k < NB; ++k)
        if (k / kH != group)
#pragma unroll
          for (int a = 0; a < NA; ++a) out[(a * kH + k % kH) * 64] = acc[a][k];
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NB; ++k)
        if (k / kH == group)
#pragma unroll
          for (int a = 0; a < NA; ++a) acc[a][k] += in[(a * kH + k % kH) * 64];
    }

    // ---------------------------------------------------------- epilogue
    // The wave stages kEpiRows rows at a time as bf16 (16-byte chunk c of row r at c ^
    // turn(r): the same chunk of sixteen rows on all banks) and stores 16-byte
    // pieces of whole row segments (a wave's LDS accesses run in order: no waits).
    {
      typedef unsigned int u4v __attribute__((ext_vector_type(4)));
      typedef u4v u4a2 __attribute__((aligned(2)));
      uint8_t* reg = smem + L::kEpiAt + (group * 4 + wave) * L::kEpiWave;
      const int nw = cur.col0 + wn * 16 * NA, mw = cur.row0 + wm * 16 * NB;
      constexpr int kLanesRow = 2 * NA, kRows = 64 / kLanesRow, kPasses = L::kEpiRows / kRows;
      const int rr = lane / kLanesRow, cc = (lane % kLanesRow) * 8;
      auto turn = [](int r) { return NA == 8 ? r & 15 : (r >> 1) & 7; };
      const int lr = li % L::kEpiRows;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        if (kGroups == 2 && k / (NB / 2) != group) continue;
#pragma unroll
        for (int part = 0; part < 16 / L::kEpiRows; ++part) {
          if (L::kEpiRows == 16 || li / L::kEpiRows == part) {
#pragma unroll
            for (int a = 0; a < NA; ++a) {
              const v4f v = acc[a][k];
              *reinterpret_cast<uint2*>(reg + lr * L::kPitch + (((2 * a + (lg >> 1)) ^ turn(lr)) << 4) +
                                        (lg & 1) * 8) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
            }
          }
          asm volatile("" ::: "memory");
          u4v o[kPasses];
#pragma unroll
          for (int r = 0; r < kPasses; ++r)
            o[r] = *reinterpret_cast<const u4v*>(reg + (rr + kRows * r) * L::kPitch +
                                                 (((cc >> 3) ^ turn(rr + kRows * r)) << 4));
#pragma unroll
          for (int r = 0; r < kPasses; ++r) {
            const int m = mw + 16 * k + L::kEpiRows * part + rr + kRows * r, n = nw + cc;
            if (m >= cur.row_end || n >= p.N) continue;
            uint16_t* d = p.y + (size_t)m * p.ldy + n;
            if (n + 7 < p.N) {
              // (the hardware serves pieces that are not on 16 bytes, too)
              if (p.past) __builtin_nontemporal_store(o[r], reinterpret_cast<u4v*>(d));
              else *reinterpret_cast<u4a2*>(d) = o[r];
            } else {
              for (int e = 0; e < 8; ++e)
                if (n + e < p.N) d[e] = (uint16_t)(o[r][e >> 1] >> (16 * (e & 1)));
            }
          }
          asm volatile("" ::: "memory");
        }
      }
    }
    if (kGroups == 2 || !nxt.live) break;
    cur = nxt;
    ++t;
  }
  // No copy may write into LDS that is no longer this workgroup's.
  tile::wait_vmcnt<0>();
}

namespace {

bool rows_on(const void* y, int64_t ldy, int64_t bytes) { return (((uintptr_t)y | (uintptr_t)(ldy * 2)) & (bytes - 1)) == 0; }

// y goes around the caches where its rows allow 16-byte pieces, but for a large
// one that a short K leaves as what counts, in parts of cache lines: those are
// better left for L2 to join (8192 x 6000 x 256 54 us around, 34 through L2; 4096
// x 6008 x 512 35 and 25, 2048 x 16008 x 1024 42 and 36; but 8192 x 6000 x 1024
// 56 and 60, 4096 x 6008 x 4096 69 and 74, and for the experts 2008 x 768, 4096
// tokens, 77 and 92).
bool past_caches(const void* y, int64_t ldy, int64_t M, int64_t N, int64_t K) {
  if (!rows_on(y, ldy, 16)) return false;
  return rows_on(y, ldy, 128) || K > (rows_on(y, ldy, 32) ? 512 : 1024) || M * N <= (int64_t)16 << 20;
}

template <int NA, int NB, int kX, bool kExperts, int kGroups = 1>
int go(const Fp4Args& p, int64_t tiles, hipStream_t stream) {
  using L = Fp4Lds<NA, NB, kX, kGroups>;
  auto kern = gemm_fp4_kernel<NA, NB, kX, kExperts, kGroups>;
  static std::atomic<int> lds_set[kMaxDevices];
  constexpr int most_lds = L::kBytes + (int)(kFp4FusedMaxK / 128) * L::kFusedStep;
  static_assert(most_lds <= 160 * 1024, "LDS of a compute unit");
  if (!set_lds_limit_once((const void*)kern, most_lds, lds_set)) return -7;
  const int lds = L::kBytes + p.K / 128 * L::kFusedStep;
  const int64_t per_cu = lds <= 80 * 1024 ? 2 : 1;
  const int64_t cus = device_cu_count();
  const int64_t most = kGroups == 2 ? tiles : std::max<int64_t>(1, (cus >= 8 ? cus - cus % 8 : cus) * per_cu);
  hipLaunchKernelGGL(kern, dim3((unsigned)std::min(tiles, most)), dim3(kThreads * kGroups), lds, stream, p);
  return hipGetLastError() == hipSuccess ? 0 : -7;
}

}  // namespace

int launch_gemm_fp4_tile(const void* qp, const void* sp, int64_t M, int64_t K, const void* wp, const void* wsp,
                         int64_t N, const void* bias, void* y, int64_t ldy, hipStream_t stream, Fp4Plan plan) {
  Fp4Args p = {};
  p.q = (const uint8_t*)qp;
  p.s = (const uint8_t*)sp;
  p.M = (int)M;
  p.K = (int)K;
  p.wp = (const uint8_t*)wp;
  p.wsp = (const uint8_t*)wsp;
  p.N = (int)N;
  p.bias = (const uint16_t*)bias;
  p.y = (uint16_t*)y;
  p.ldy = ldy;
  p.past = past_caches(y, ldy, M, N, K);
  const int64_t tiles = ((M + plan.mt - 1) / plan.mt) * ((N + plan.nt - 1) / plan.nt);
  if (plan.nt == 256) return go<8, 8, kPacked, false>(p, tiles, stream);
  // One tile per compute unit: two groups of waves; more: two workgroups on each.
  const bool one = tiles <= device_cu_count();
  if (plan.mt == 128)
    return one ? go<4, 4, kPacked, false, 2>(p, tiles, stream) : go<4, 4, kPacked, false>(p, tiles, stream);
  return one ? go<4, 2, kPacked, false, 2>(p, tiles, stream) : go<4, 2, kPacked, false>(p, tiles, stream);
}

int launch_experts_fp4_tile(const ExpertsArgs& a, const void* q, const void* s, Fp4Plan plan, hipStream_t stream) {
  Fp4Args p = {};
  p.q = (const uint8_t*)q;
  p.s = (const uint8_t*)s;
  p.q_bytes = (uint32_t)(a.x_rows * (a.K / 2));
  p.s_pitch = (uint32_t)fp4_scale_pitch(a.K);
  p.s_bytes = (uint32_t)(a.x_rows * fp4_scale_pitch(a.K));
  p.K = (int)a.K;
  p.wp = (const uint8_t*)a.wp;
  p.wsp = (const uint8_t*)a.wsp;
  p.N = (int)a.N;
  p.y = (uint16_t*)a.y;
  p.ldy = a.ldy;
  p.past = rows_on(a.y, a.ldy, 16);
  p.R = (int)a.R;
  p.E = (int)a.E;
  p.topk = (int)a.topk;
  p.slots = a.slots;
  p.offsets = a.offsets;
  // At most one more row tile per expert than the rows fill.
  const int64_t row_tiles = a.R / plan.mt + std::min(a.E, a.R);
  const int64_t tiles = row_tiles * ((a.N + plan.nt - 1) / plan.nt);
  if (plan.nt == 256) return go<8, 4, kRows, true>(p, tiles, stream);
  if (plan.mt == 128) return go<4, 4, kRows, true>(p, tiles, stream);
  return go<4, 2, kRows, true>(p, tiles, stream);
}

int launch_gemm_fp4_fused(const void* x, int64_t ldx, int64_t M, int64_t K, const void* wp, const void* wsp, int64_t N,
                          const void* bias, void* y, int64_t ldy, hipStream_t stream) {
  Fp4Args p = {};
  p.x = (const uint16_t*)x;
  p.ldx = ldx;
  p.x_rows = (int)M;
  p.M = (int)M;
  p.K = (int)K;
  p.wp = (const uint8_t*)wp;
  p.wsp = (const uint8_t*)wsp;
  p.N = (int)N;
  p.bias = (const uint16_t*)bias;
  p.y = (uint16_t*)y;
  p.ldy = ldy;
  p.past = past_caches(y, ldy, M, N, K);
  const int64_t tiles = (M + 63) / 64 * ((N + 127) / 128);
  return tiles <= device_cu_count() ? go<4, 2, kFused, false, 2>(p, tiles, stream)
                                    : go<4, 2, kFused, false>(p, tiles, stream);
}

int launch_experts_fp4_fused(const ExpertsArgs& a, hipStream_t stream) {
  Fp4Args p = {};
  p.x = (const uint16_t*)a.x;
  p.ldx = a.ldx;
  p.x_rows = (int)a.x_rows;
  p.K = (int)a.K;
  p.wp = (const uint8_t*)a.wp;
  p.wsp = (const uint8_t*)a.wsp;
  p.N = (int)a.N;
  p.y = (uint16_t*)a.y;
  p.ldy = a.ldy;
  p.past = rows_on(a.y, a.ldy, 16);
  p.R = (int)a.R;
  p.E = (int)a.E;
  p.topk = (int)a.topk;
  p.slots = a.slots;
  p.offsets = a.offsets;
  const int64_t tiles = (a.R / 64 + std::min(a.E, a.R)) * ((a.N + 127) / 128);
  return tiles <= device_cu_count() ? go<4, 2, kFused, true, 2>(p, tiles, stream)
                                    : go<4, 2, kFused, true>(p, tiles, stream);
}

}  // namespace mxfp8
