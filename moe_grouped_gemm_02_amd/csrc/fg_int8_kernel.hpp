// fg_int8_kernel.hpp -- gfx950 kernels of the 8-bit integer product
//
//     D[m, n] = bf16( sa[m] sb[n] sum_k A[m, k] B[n, k] )
//
// in the dense, contiguous and masked layouts. The sum runs in 32-bit integers on
// the matrix core (v_mfma_i32_16x16x64_i8) and is exact: 128^2 K < 2^31 up to K =
// 131071, so the result does not depend on tile, layout or order; the only
// roundings are the sum's to fp32 (24 bits), the two scales' products in fp32 and
// the last one to bf16.
//
// The tiles move as the E4M3 kernels' do (fg_kernel.hpp: global->LDS DMA into
// XOR-swizzled rings, loads spread over the MFMAs, B rows in pair_column order for
// 16-byte stores straight from the accumulators, the next tile's first loads before
// this tile's stores) and share those helpers. What differs: one scale per row and
// column means nothing is promoted in the K loop, every MFMA accumulates in place;
// a tile's scales come once, into an LDS slot of their own, and are applied in the
// epilogue; and K is any multiple of 16: the chunks of the last K-block past K get
// offsets past the buffer and read as zeros.
//
// What bounds it, measured on one MI355X: 8192 x 7168 x 18432 takes 726-750 us (2.9-3.0
// POP/s; this instruction alone, on normal random codes in registers, 4.2, on zeros 4.9, the
// 32x32x32 form 3.5). The matrix cores are busy 74-78% of the cycles -- the rest are a K-block's
// two barriers and the tiles' ends -- and the clock is 1.8-1.9 GHz, where the instruction alone
// has 2.0. 8 experts contiguous (8192 rows, N 4096, K 7168) 220-228 us, the same in 2.3 rounds of
// tiles. 16 experts masked (M_max 256, N 7168, K 2048) 67-70 us: the stream of the weights through
// those barriers, 3.4 TB/s of them (3.9 of all that moves); 256x224 tiles 68, 128-row tiles 80-88.
#pragma once

#include "fg_kernel.hpp"
#include "fg_wave.hpp"

namespace fg {

// Compile-time tile configuration: as TileCfg, without scales in the rings.
template <int BM_, int BN_, int WGM_, int WGN_, int STAGES_, int PD_>
struct Int8Cfg {
  static constexpr int BM = BM_, BN = BN_, WGM = WGM_, WGN = WGN_, STAGES = STAGES_;
  static constexpr int PD = PD_, RING = PD_ + 1;
  static constexpr int W = WGM * WGN, THREADS = 64 * W;
  static constexpr int WM = BM / WGM, WN = BN / WGN, TM = WM / 16, TN = WN / 16;
  static constexpr int A_INSTR = (BM * 8 + 64 * W - 1) / (64 * W);
  static constexpr int B_INSTR = (BN * 8 + 64 * W - 1) / (64 * W);
  static constexpr int DMA_PER_STAGE = A_INSTR + B_INSTR;
  static constexpr int A_BYTES = A_INSTR * W * 1024, B_BYTES = B_INSTR * W * 1024;
  // two slots of a tile's scales (this tile's and the next one's), then the rings
  static constexpr int SC_LOADS = BM / 64 + (BN + 63) / 64;   // 64 scales a load
  static constexpr int SC_BYTES = SC_LOADS * 256;
  static constexpr int A_BASE = 2 * SC_BYTES;
  static constexpr int B_BASE = A_BASE + STAGES * A_BYTES;
  static constexpr int LDS_BYTES = B_BASE + STAGES * B_BYTES;
  static constexpr int UNROLL = lcm_c(STAGES, RING / gcd_c(TN, RING));
  static_assert(WM % 16 == 0 && WN % 32 == 0 && BM % 64 == 0, "whole sub-tile pairs, scales 64 at a time");
  static_assert(BM % WGM == 0 && BN % WGN == 0, "waves must split the tile evenly");
  static_assert(STAGES >= 2, "ring depth");
  static_assert(STAGES * DMA_PER_STAGE <= 63, "too many DMA instructions in flight per wave");
  static_assert(LDS_BYTES <= 160 * 1024, "LDS exceeds 160 KB");
  static_assert(PD >= 1 && PD <= TN - 1, "prefetch distance must leave the barrier inside the K-block");
};

__device__ __forceinline__ i32x4 mfma_i8(const i32x4& b, const i32x4& a, const i32x4& acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(b, a, acc, 0, 0, 0);
}
__device__ __forceinline__ i32x4 mfma_i8_lo(const i32x8& b, const i32x8& a, const i32x4& acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(i32x4{b[0], b[1], b[2], b[3]}, i32x4{a[0], a[1], a[2], a[3]}, acc, 0, 0, 0);
}
__device__ __forceinline__ i32x4 mfma_i8_hi(const i32x8& b, const i32x8& a, const i32x4& acc) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(i32x4{b[4], b[5], b[6], b[7]}, i32x4{a[4], a[5], a[6], a[7]}, acc, 0, 0, 0);
}
// One step: its two MFMAs, its LDS reads, then the rest; nothing crosses steps.
__device__ __forceinline__ void int8_step_fence() {
  __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
  __builtin_amdgcn_sched_group_barrier(0x100, 8, 0);
  __builtin_amdgcn_sched_group_barrier(0x002, 16, 0);
  __builtin_amdgcn_sched_barrier(0);
}

// The tiles a workgroup computes one after another: next(d) fills the next one and
// returns true, or returns false (uniform over the workgroup).
template <int LAYOUT, class T, class Next>
__device__ __forceinline__ void int8_tiles(const Params& p, lds_u8* const lds, Next&& next) {
  constexpr int BM = T::BM, BN = T::BN, W = T::W, WM = T::WM, WN = T::WN;
  constexpr int TM = T::TM, TN = T::TN, PD = T::PD, R = T::RING, NA = T::A_INSTR, NB = T::B_INSTR;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = uniform(t >> 6);
  const int wm = wave / T::WGN, wn = wave % T::WGN;
  const int lr = lane & 15, lq = lane >> 4;
  const int K = p.K, nkb = p.KB, M = p.M;
  const uint32_t lds_addr = (uint32_t)(uintptr_t)lds;
  const uint32_t wave_at = lds_addr + wave * 1024;

  auto next_tile = [&](TileDesc& d) {
    const bool more = uniform(next(d) ? 1 : 0) != 0;
    d = TileDesc{uniform(d.g), uniform(d.m0), uniform(d.n0), uniform(d.rows_valid)};
    return more;
  };
  TileDesc cur;
  if (!next_tile(cur)) return;

  // DMA lane sources: slot s of a tile region is its 16-byte chunk s, holding row s / 8,
  // chunk (s % 8) ^ (row % 8); a lane's chunk is the same for all its instructions.
  const uint32_t chunk16 = (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16);
  uint32_t a_off[NA], b_off[NB];
  auto a_row = [&](int q) { return ((q * W + wave) * 64 + lane) >> 3; };
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const int row = a_row(q);
    a_off[q] = row < BM ? (uint32_t)row * (uint32_t)K + chunk16 : kNoRow;
  }
#pragma unroll
  for (int q = 0; q < NB; ++q) {
    const int row = a_row(q);
    b_off[q] = row < BN ? (uint32_t)pair_column(row) * (uint32_t)K + chunk16 : kNoRow;
  }
  i32x4 rsA, rsB;
  constexpr int NWIN = (T::LDS_BYTES + 65535) >> 16;
  LdsAddr<NWIN> aLo, aHi, bLo, bHi;
  {
    const uint32_t lane_lo = lr * 128 + ((lq ^ (lr & 7)) << 4);
    const uint32_t lane_hi = lr * 128 + (((lq + 4) ^ (lr & 7)) << 4);
    aLo.init(lds_addr + wm * WM * 128 + lane_lo);
    aHi.init(lds_addr + wm * WM * 128 + lane_hi);
    bLo.init(lds_addr + wn * WN * 128 + lane_lo);
    bHi.init(lds_addr + wn * WN * 128 + lane_hi);
  }
  // Resources of tile d; rows past its last row with an output and columns past N read
  // zeros. Its scales go to LDS slot par: loads older than the tile's first stage, so
  // the wait for that stage covers them.
  auto setup = [&](const TileDesc& d, int par) {
    const int g = d.g, m0 = d.m0, n0 = d.n0;
    const uint8_t* Ag = p.A + (LAYOUT == kMasked ? (size_t)g * M * K : 0);
    const float* sag = p.sa + (LAYOUT == kMasked ? (size_t)g * M : 0);
    const uint8_t* Bg = p.B + (LAYOUT != kDense ? (size_t)g * p.N * K : 0);
    const float* sbg = p.sb + (LAYOUT != kDense ? (size_t)g * p.N : 0);
    const int rows = max(0, min(d.rows_valid - m0, BM)), cols = max(0, min(p.N - n0, BN));
    rsA = buffer_rsrc(Ag + (size_t)m0 * K, (uint32_t)rows * (uint32_t)K);
    rsB = buffer_rsrc(Bg + (size_t)n0 * K, (uint32_t)cols * (uint32_t)K);
    const i32x4 rsSA = buffer_rsrc(sag + m0, (uint32_t)rows * 4u), rsSB = buffer_rsrc(sbg + n0, (uint32_t)cols * 4u);
    if constexpr (LAYOUT == kContiguous) {
      // rows of padding or of another expert load nothing
#pragma unroll
      for (int q = 0; q < NA; ++q) {
        const int row = a_row(q), m = m0 + row;
        const bool live = row < BM && m < M && p.m_indices[m] == g;
        a_off[q] = live ? (uint32_t)row * (uint32_t)K + chunk16 : kNoRow;
        asm volatile("" : "+v"(a_off[q]));   // its load completes before the DMAs below
      }
    }
    const uint32_t at = lds_addr + par * T::SC_BYTES;
#pragma unroll
    for (int q = 0; q < (T::SC_LOADS + W - 1) / W; ++q) {
      const int i = q * W + wave;
      if (i < BM / 64) dma4<0>(rsSA, (uint32_t)(i * 64 + lane) * 4u, 0u, at + i * 256);
      else if (i < T::SC_LOADS) dma4<0>(rsSB, (uint32_t)((i - BM / 64) * 64 + lane) * 4u, 0u, at + i * 256);
    }
  };
  // Scalar offset of the DMAs of K-block kb (or of the last one), and what puts a lane's
  // chunk past the buffer where it lies past K.
  struct Soff {
    uint32_t at, past;
  };
  auto soff_of = [&](int kb) {
    const uint32_t at = (uint32_t)min(kb, nkb - 1) * (uint32_t)kKBlock;
    return Soff{at, at + chunk16 >= (uint32_t)K ? kNoRow : 0u};
  };
  auto issue = [&](auto d_c, auto st_c, const Soff& o) {
    constexpr int d = decltype(d_c)::value, ST = decltype(st_c)::value;
    if constexpr (d < NA) dma16<T::A_BASE + ST * T::A_BYTES + d * W * 1024>(rsA, a_off[d] | o.past, o.at, wave_at);
    else dma16<T::B_BASE + ST * T::B_BYTES + (d - NA) * W * 1024>(rsB, b_off[d - NA] | o.past, o.at, wave_at);
  };
  auto fragA = [&](auto st_c, auto i_c) {
    return frag_at<T::A_BASE + decltype(st_c)::value * T::A_BYTES + decltype(i_c)::value * 2048>(aLo, aHi);
  };
  auto fragB = [&](auto st_c, auto j_c) {
    return frag_at<T::B_BASE + decltype(st_c)::value * T::B_BYTES + decltype(j_c)::value * 2048>(bLo, bHi);
  };

  // DMA schedule: that of gemm_tiles (fg_kernel.hpp), which states why each wait suffices.
  using SCH = Sched<T>;
  constexpr int STEPS = SCH::STEPS, PRE = SCH::PRE, POST = SCH::POST, D = SCH::D;
  constexpr bool SPLIT = SCH::SPLIT;
  constexpr int S = T::STAGES;
  constexpr int WAIT_LOOP = SPLIT ? SCH::n_early() : (S - 2) * D;
  constexpr int WAIT_PRO = SPLIT ? D : (S - 2) * D + SCH::n_head();
  constexpr int NST = TM * (TN / 2);   // output stores per wave and tile
  static_assert(WAIT_PRO + NST < 64 && WAIT_LOOP < 64, "vmcnt counter range");
  auto prologue = [&]() {
    static_for<S>([&](auto x_c) {
      constexpr int x = decltype(x_c)::value;
      const Soff o = soff_of(x);
      static_for<D>([&](auto d_c) {   // S >= 3: the rest of the last stage comes with the first K-block
        if constexpr (SPLIT || x != S - 1 || SCH::slot(decltype(d_c)::value) < POST) issue(d_c, x_c, o);
      });
    });
  };
  int par = 0;
  setup(cur, par);
  prologue();
  TileDesc nx = cur;
  bool after_stores = false;
  for (;;) {
    if (after_stores) wait_vm<WAIT_PRO + NST>();
    else wait_vm<WAIT_PRO>();
    block_barrier();
    i32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
      for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
    i32x8 fbr[R], fa[TM];
    {
      using Z = std::integral_constant<int, 0>;
      static_for<PD>([&](auto c_c) {
        fbr[decltype(c_c)::value] = fragB(Z{}, c_c);
        __builtin_amdgcn_sched_barrier(0);
      });
      static_for<TM>([&](auto i_c) {
        fa[decltype(i_c)::value] = fragA(Z{}, i_c);
        __builtin_amdgcn_sched_barrier(0);
      });
    }
    int kb = 0;
    auto kblock = [&](auto ph_c) -> bool {
      constexpr int PH = decltype(ph_c)::value, U = T::UNROLL;
      using Cur = std::integral_constant<int, PH % S>;
      using Nxt = std::integral_constant<int, (PH + 1) % S>;
      using Tail = std::integral_constant<int, (PH + U - 1) % S>;
      const Soff head = soff_of(kb + S), tail = soff_of(kb - 1 + S);
      (void)tail;
      static_for<STEPS>([&](auto u_c) {
        constexpr int u = decltype(u_c)::value, j = u / TM, i = u % TM;
        if constexpr (SPLIT && u == TM && TM < PRE) block_barrier();   // A half of this stage is free
        if constexpr (u == PRE) {
          wait_lgkm0();
          wait_vm<WAIT_LOOP>();
          block_barrier();
        }
        acc[i][j] = mfma_i8_lo(fbr[(PH * TN + j) % R], fa[i], acc[i][j]);
        acc[i][j] = mfma_i8_hi(fbr[(PH * TN + j) % R], fa[i], acc[i][j]);
        if constexpr (i == 0) {
          constexpr int jn = j + PD, slot = (PH * TN + jn) % R;
          if constexpr (jn < TN) fbr[slot] = fragB(Cur{}, std::integral_constant<int, jn>{});
          else fbr[slot] = fragB(Nxt{}, std::integral_constant<int, jn - TN>{});
        }
        if constexpr (j == TN - 1) fa[i] = fragA(Nxt{}, std::integral_constant<int, i>{});
        static_for<D>([&](auto d_c) {
          constexpr int d = decltype(d_c)::value;
          if constexpr (SPLIT) {
            if constexpr (SCH::slot(d) == u) issue(d_c, Cur{}, head);
          } else {
            if constexpr (u >= PRE && SCH::slot(d) == u - PRE) issue(d_c, Cur{}, head);
            if constexpr (u < PRE && SCH::slot(d) == POST + u) issue(d_c, Tail{}, tail);
          }
        });
        int8_step_fence();
      });
      return ++kb == nkb;
    };
    bool done = false;
    for (;;) {
      static_for<T::UNROLL>([&](auto ph_c) {
        if (!done) done = kblock(ph_c);
      });
      if (done) break;
    }

    const int g = cur.g, m0 = cur.m0, n0 = cur.n0, rows_valid = cur.rows_valid;
    uint16_t* Dg = p.D + (LAYOUT == kMasked ? (size_t)g * M * p.N : 0);
    wait_vm<0>();          // the clamped tail DMAs must land before LDS is reused
    wait_lgkm0();
    block_barrier();
    const int rows_here = max(0, min(rows_valid - m0, BM));
    const __amdgpu_buffer_rsrc_t rsD =
        __builtin_amdgcn_make_buffer_rsrc(Dg + (size_t)m0 * p.N, 0, rows_here * p.N * 2, 0x20000);
    const lds_u8* sc = lds + par * T::SC_BYTES;
    uint32_t roff[TM];
    float sa[TM];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      const int ml = wm * WM + i * 16 + lr, m = m0 + ml;
      bool ok = m < rows_valid;
      if (LAYOUT == kContiguous && ok) ok = p.m_indices[m] == g;
      roff[i] = ok ? (uint32_t)ml * (uint32_t)p.N * 2u : kNoRow;
      asm volatile("" : "+v"(roff[i]));   // any m_indices load completes before the next tile's DMAs
      sa[i] = *(const lds_f32*)(sc + ml * 4);
    }
    const bool more = next_tile(nx);
    if (more) {
      setup(nx, par ^ 1);
      prologue();
    }
#pragma unroll
    for (int q = 0; q < TN / 2; ++q) {
      const int nl = wn * WN + q * 32 + lq * 8, n = n0 + nl;
      typedef __attribute__((address_space(3))) const f32x4 lds_f32x4c;
      const f32x4 s0 = *(lds_f32x4c*)(sc + (BM + nl) * 4), s1 = *(lds_f32x4c*)(sc + (BM + nl) * 4 + 16);
#pragma unroll
      for (int i = 0; i < TM; ++i) {
        const uint32_t off = n < p.N ? roff[i] + (uint32_t)n * 2u : kNoRow;
        const i32x4& x = acc[i][2 * q];
        const i32x4& y = acc[i][2 * q + 1];
        float f[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          f[c] = (float)x[c] * sa[i] * s0[c];
          f[4 + c] = (float)y[c] * sa[i] * s1[c];
        }
        const i32x4 v = {(int)bf16_pair(f[0], f[1]), (int)bf16_pair(f[2], f[3]), (int)bf16_pair(f[4], f[5]),
                         (int)bf16_pair(f[6], f[7])};
        __builtin_amdgcn_raw_buffer_store_b128(v, rsD, off, 0, 0);
      }
    }
    if (!more) break;
    cur = nx;
    par ^= 1;
    after_stores = true;
  }
}

// One tile per workgroup.
template <int LAYOUT, class T>
__global__ __launch_bounds__(T::THREADS) void int8_gemm(Params p) {
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS_BYTES];
  __shared__ int s_group;
  lds_u8* const lds = (lds_u8*)smem;
  const int t = threadIdx.x;
  int tile = xcd_position(blockIdx.x, gridDim.x);
  int g = 0;
  if (LAYOUT == kMasked) {
    const int per = p.tiles_m * p.tiles_n;
    g = tile / per;
    tile -= g * per;
  }
  int mb, nbk;
  raster(tile, p.tiles_m, p.tiles_n, mb, nbk);
  const int m0 = mb * T::BM, n0 = nbk * T::BN;
  int rows_valid = p.M;
  if (LAYOUT == kMasked) {
    const int mm = p.masked_m[g];
    rows_valid = mm < 0 ? 0 : (mm > p.M ? p.M : mm);
    if (m0 >= rows_valid) return;   // uniform over the workgroup
  }
  if (LAYOUT == kContiguous) {
    if (t == 0) s_group = -1;
    __syncthreads();
    if (t < T::BM && m0 + t < p.M) {
      const int id = p.m_indices[m0 + t];
      if (id >= 0 && id < p.G) atomicMax(&s_group, id);
    }
    __syncthreads();
    g = s_group;
    if (g < 0) return;   // all-padding block
  }
  bool done = false;
  int8_tiles<LAYOUT, T>(p, lds, [&](TileDesc& d) {
    if (done) return false;
    d = TileDesc{g, m0, n0, rows_valid};
    done = true;
    return true;
  });
}

// Dense on two tile shapes, contiguous on run-following tiles: the schedules of
// fp8_bs_gemm_split and fp8_bs_gemm_runs.
template <class TA, class TB>
__global__ __launch_bounds__(TA::THREADS) void int8_gemm_split(Params p) {
  static_assert(TA::THREADS == TB::THREADS, "both tile shapes run with the same workgroup size");
  constexpr int LDS = TA::LDS_BYTES > TB::LDS_BYTES ? TA::LDS_BYTES : TB::LDS_BYTES;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS];
  lds_u8* const lds = (lds_u8*)smem;
  const int grid = gridDim.x, na = p.tiles_a;
  const int tma = (p.M + TA::BM - 1) / TA::BM, tna = p.n_split / TA::BN;
  const int tmb = (p.M + TB::BM - 1) / TB::BM, tnb = (p.N - p.n_split + TB::BN - 1) / TB::BN;
  const int nb = tmb * tnb;
  int k = blockIdx.x;
  int8_tiles<kDense, TA>(p, lds, [&](TileDesc& d) {
    if (k >= na) return false;
    int mb, nbk;
    raster(xcd_position(k, na), tma, tna, mb, nbk);
    d = TileDesc{0, mb * TA::BM, nbk * TA::BN, p.M};
    k += grid;
    return true;
  });
  wait_lgkm0();
  block_barrier();   // no wave still reads the TA tiles' LDS when the TB tiles' DMAs start
  k = blockIdx.x;
  int8_tiles<kDense, TB>(p, lds, [&](TileDesc& d) {
    if (k >= nb) return false;
    int mb, nbk;
    raster(xcd_position(k, nb), tmb, tnb, mb, nbk);
    d = TileDesc{0, mb * TB::BM, p.n_split + nbk * TB::BN, p.M};
    k += grid;
    return true;
  });
}

// Where the last round's single-block tiles leave three of four workgroups idle, it runs as quarters
// of them (8192 rows of 8 experts, N 4096, K 7168: 233 to 226 us).
template <class TF, class TH, class TQ>
__global__ __launch_bounds__(TF::THREADS) void int8_gemm_runs(Params p) {
  static_assert(TF::BM == 256 && TH::BM == 128 && TF::BN == TH::BN && TF::THREADS == TH::THREADS,
                "two-block tiles of 256 rows, single-block tiles of 128 rows, same columns and workgroup");
  static_assert(TQ::BM == 64 && 2 * TQ::BN == TH::BN && TQ::THREADS == TH::THREADS, "quarters of a single-block tile");
  static_assert(TQ::LDS_BYTES <= TH::LDS_BYTES, "LDS of the larger tiles");
  constexpr int LDS = TF::LDS_BYTES > TH::LDS_BYTES ? TF::LDS_BYTES : TH::LDS_BYTES;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[LDS + kRunMaxBlocks * 4];
  __shared__ int s_count[2];
  lds_u8* const lds = (lds_u8*)smem;
  int* list = (int*)(smem + LDS);
  contiguous_run_tiles<TF::THREADS, true>(p, (int*)smem, list, s_count);
  const int F = s_count[0], S = s_count[1], tn = p.tiles_n;
  const long grid = gridDim.x;
  const long full_items = (long)F * tn;
  long whole = full_items;   // two-block tiles that run as 256-row tiles
  {
    const long rounds = full_items / grid, rest = full_items - rounds * grid;
    if (rest && 2 * rest + (long)S * tn <= grid) whole = rounds * grid;
  }
  const long halves = 2 * (full_items - whole);
  const long items = whole + halves + (long)S * tn;
  const long last = items % grid;
  const long quartered = last <= items - whole && 4 * last <= grid ? last : 0;   // the last round's
  long w = xcd_position(blockIdx.x, gridDim.x);
  int8_tiles<kContiguous, TF>(p, lds, [&](TileDesc& d) {
    if (w >= whole) return false;
    int mb, nbk;
    raster((int)w, F, tn, mb, nbk);
    const int e = list[mb];
    d = TileDesc{e >> 16, (e & 0xffff) * 128, nbk * TF::BN, p.M};
    w += grid;
    return true;
  });
  wait_lgkm0();
  block_barrier();   // no wave still reads LDS of the 256-row tiles when the 128-row ones start
  auto single = [&](long h) {
    int mb, nbk, e, m0;
    if (h < halves) {   // one 128-row half of a two-block tile
      raster((int)(whole + h / 2), F, tn, mb, nbk);
      e = list[mb];
      m0 = (e & 0xffff) * 128 + (int)(h & 1) * 128;
    } else {            // a single-block tile
      raster((int)(h - halves), S, tn, mb, nbk);
      e = list[kRunMaxBlocks - 1 - mb];
      m0 = (e & 0xffff) * 128;
    }
    return TileDesc{e >> 16, m0, nbk * TH::BN, p.M};
  };
  int8_tiles<kContiguous, TH>(p, lds, [&](TileDesc& d) {
    if (w >= items - quartered) return false;
    d = single(w - whole);
    w += grid;
    return true;
  });
  // items - quartered are whole rounds: what is left of w is this workgroup's quarter
  long q = w - (items - quartered);
  if (q >= 4 * quartered) return;   // uniform over the workgroup
  wait_lgkm0();
  block_barrier();
  int8_tiles<kContiguous, TQ>(p, lds, [&](TileDesc& d) {
    if (q < 0) return false;
    d = single(items - quartered - whole + q / 4);
    d.m0 += (int)(q & 1) * TQ::BM;
    d.n0 += (int)(q >> 1 & 1) * TQ::BN;
    q = -1;
    return d.n0 < p.N && d.m0 < p.M;
  });
}

// Few rows or few columns: the product is a stream of its operands. A workgroup has 16 TN columns and
// 16 TM rows, so few that all CUs have some; its waves take 128-byte pieces of K in turn and add their sums up
// through LDS at the end -- exact in any order, so K needs no split over workgroups and no
// workspace. Each wave moves its pieces through a ring of STAGES slots of its own in LDS
// (whole 128-byte lines a load; straight into the matrix core's registers a load takes 16
// half lines, which the CU fetches at a third of the rate: M 64, N 7168, K 7168 22.7 us),
// so nothing but the end needs a barrier: 9.5-10 us and 12 us for 16 and 64 rows, the weights
// at 5.4 TB/s in the first, launch included. Chunks past the last row, column or K get
// offsets past the buffer: zeros, and no memory access.
template <int TM_, int TN_, int WAVES_, int STAGES_>
struct SkinnyCfg {
  static constexpr int TM = TM_, TN = TN_, WAVES = WAVES_, STAGES = STAGES_;
  static constexpr int LOADS = 2 * (TM + TN);                   // of a piece, a kilobyte each
  static constexpr int RING = STAGES * LOADS * 1024;            // of a wave
  static constexpr int BLOCKS = (TM * TN + WAVES - 1) / WAVES;  // 16x16 blocks of D a wave finishes
  static constexpr int LDS_BYTES = WAVES * RING > WAVES * TM * TN * 1024 ? WAVES * RING : WAVES * TM * TN * 1024;
  static_assert(LDS_BYTES <= 160 * 1024 && STAGES * LOADS < 48, "LDS and the loads in flight");
};
template <int LAYOUT, class T>
__global__ __launch_bounds__(64 * T::WAVES) void int8_skinny(Params p) {
  constexpr int TM = T::TM, TN = T::TN, W = T::WAVES, S = T::STAGES, U = T::BLOCKS;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS_BYTES];
  lds_u8* const lds = (lds_u8*)smem;
  const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = uniform(threadIdx.x >> 6);
  // row blocks of the same columns follow one another on one XCD, whose L2 has the weights then
  int g = 0, tile = p.tiles_m == 1 ? blockIdx.x : xcd_position(blockIdx.x, gridDim.x);
  if (LAYOUT == kMasked) {
    const int per = p.tiles_m * p.tiles_n;
    g = tile / per;
    tile -= g * per;
  }
  const int n0 = tile / p.tiles_m * 16 * TN, m0 = tile % p.tiles_m * 16 * TM;
  int rows = p.M;
  if (LAYOUT == kMasked) {
    const int mm = p.masked_m[g];
    rows = mm < 0 ? 0 : (mm > p.M ? p.M : mm);
    if (m0 >= rows) return;   // uniform over the workgroup
  }
  rows = min(rows - m0, 16 * TM);
  const int K = p.K, cols = min(p.N - n0, 16 * TN);
  if (LAYOUT == kContiguous) {   // the expert of these rows' block of 128; every wave looks it up for itself
    static_assert(LAYOUT != kContiguous || 8 % TM == 0, "blocks of rows within one of 128");
    int top = -1;
#pragma unroll
    for (int r = 0; r < 16 * TM; r += 64) {
      const int id = r + lane < rows ? p.m_indices[m0 + r + lane] : -1;
      if (id >= 0 && id < p.G) top = max(top, id);
    }
    g = (int)group_max_u32<64>((uint32_t)(top + 1)) - 1;
    if (g < 0) return;   // padding only; uniform over the workgroup
  }
  const size_t row0 = (LAYOUT == kMasked ? (size_t)g * p.M : 0) + m0;   // of A, sa and D
  const uint8_t* Ag = p.A + row0 * K;
  const uint8_t* Bg = p.B + ((LAYOUT != kDense ? (size_t)g * p.N : 0) + (size_t)n0) * K;
  const float* sag = p.sa + row0;
  const float* sbg = p.sb + (LAYOUT != kDense ? (size_t)g * p.N : 0);
  // the scales of the D that this lane finishes
  float sa[U], sb[U][4];
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const int u = min(wave + c * W, TM * TN - 1);
    sa[c] = sag[min(u / TN * 16 + lr, rows - 1)];
#pragma unroll
    for (int e = 0; e < 4; ++e) sb[c][e] = sbg[min(n0 + u % TN * 16 + lq * 4 + e, p.N - 1)];
  }
#pragma unroll
  for (int c = 0; c < U; ++c) {   // loaded before the first DMA: a wait for them is none for the stream
    asm volatile("" : "+v"(sa[c]), "+v"(sb[c][0]), "+v"(sb[c][1]), "+v"(sb[c][2]), "+v"(sb[c][3]));
  }
  const i32x4 rsA = buffer_rsrc(Ag, (uint32_t)rows * (uint32_t)K), rsB = buffer_rsrc(Bg, (uint32_t)cols * (uint32_t)K);
  // A load brings 8 rows: lane l chunk (l % 8) ^ (l / 8) of row l / 8, to 16-byte slot l.
  const uint32_t chunk16 = (uint32_t)(((lane & 7) ^ (lane >> 3)) * 16), row_off = (uint32_t)(lane >> 3) * (uint32_t)K + chunk16;
  const uint32_t ring = (uint32_t)(uintptr_t)lds + wave * T::RING;
  uint32_t no_row[LAYOUT == kContiguous ? 2 * TM : 1] = {};   // kNoRow for rows of padding or of another expert
  if (LAYOUT == kContiguous) {
#pragma unroll
    for (int q = 0; q < 2 * TM; ++q) {
      const int row = 8 * q + (lane >> 3);
      no_row[q] = row < rows && p.m_indices[m0 + row] == g ? 0u : kNoRow;
      asm volatile("" : "+v"(no_row[q]));   // its load completes before the DMAs
    }
  }
  auto load = [&](uint32_t slot, int x) {
    const uint32_t k = (uint32_t)(x * W + wave) * 128u;
    const uint32_t off = row_off | (k + chunk16 < (uint32_t)K ? 0u : kNoRow), step = 8u * (uint32_t)K;
    const uint32_t at = min(k, (uint32_t)K);   // within the buffer, of at least one row
    static_for<2 * TM>([&](auto q) {
      constexpr int n = decltype(q)::value;
      dma16<n * 1024>(rsA, (off + n * step) | no_row[LAYOUT == kContiguous ? n : 0], at, ring + slot);
    });
    static_for<2 * TN>([&](auto q) {
      dma16<(2 * TM + decltype(q)::value) * 1024>(rsB, off + decltype(q)::value * step, at, ring + slot);
    });
  };
  i32x4 acc[TM][TN];
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  const lds_u8* const mine = lds + wave * T::RING + lr * 128;
  const int lo = (lq ^ (lr & 7)) << 4, hi = ((lq + 4) ^ (lr & 7)) << 4;
  // A slot's piece into registers, the slot's next one on its way (if any), the products.
  auto piece = [&](uint32_t slot, int next) {
    typedef __attribute__((address_space(3))) const i32x4 lds_i32x4;
    i32x4 a[TM][2], b[TN][2];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
      a[i][0] = *(lds_i32x4*)(mine + slot + i * 2048 + lo);
      a[i][1] = *(lds_i32x4*)(mine + slot + i * 2048 + hi);
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      b[j][0] = *(lds_i32x4*)(mine + slot + (TM + j) * 2048 + lo);
      b[j][1] = *(lds_i32x4*)(mine + slot + (TM + j) * 2048 + hi);
    }
    if (next >= 0) {
      wait_lgkm0();
      load(slot, next);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = mfma_i8(b[j][h], a[i][h], acc[i][j]);
  };
  const int pieces = (K + 128 * W - 1) / (128 * W);   // of a wave
  static_for<S>([&](auto s) { load(decltype(s)::value * T::LOADS * 1024, decltype(s)::value); });
  uint32_t slot = 0;
  auto advance = [&]() { slot = slot == (S - 1) * T::LOADS * 1024 ? 0 : slot + T::LOADS * 1024; };
  for (int x = 0; x + S < pieces; ++x) {
    wait_vm<(S - 1) * T::LOADS>();
    piece(slot, x + S);
    advance();
  }
  static_for<S>([&](auto s) {
    wait_vm<(S - 1 - decltype(s)::value) * T::LOADS>();
    piece(slot, -1);
    advance();
  });
  wait_lgkm0();
  block_barrier();   // the rings are free
  typedef __attribute__((address_space(3))) i32x4 lds_i32x4w;
  lds_i32x4w* sums = (lds_i32x4w*)lds;
#pragma unroll
  for (int i = 0; i < TM; ++i)
#pragma unroll
    for (int j = 0; j < TN; ++j) sums[(wave * TM * TN + i * TN + j) * 64 + lane] = acc[i][j];
  wait_lgkm0();
  block_barrier();
  uint16_t* Dg = p.D + row0 * p.N;
#pragma unroll
  for (int c = 0; c < U; ++c) {
    const int u = wave + c * W;
    if (u >= TM * TN) break;
    const int m = u / TN * 16 + lr, n = n0 + u % TN * 16 + lq * 4;
    i32x4 v = sums[u * 64 + lane];
#pragma unroll
    for (int w = 1; w < W; ++w) v += sums[(w * TM * TN + u) * 64 + lane];
    if (m >= rows || n >= p.N) continue;
    if (LAYOUT == kContiguous && p.m_indices[m0 + m] != g) continue;
    float f[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = (float)v[e] * sa[c] * sb[c][e];
    *(u32x2*)(Dg + (size_t)m * p.N + n) = u32x2{bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3])};
  }
}

}  // namespace fg
