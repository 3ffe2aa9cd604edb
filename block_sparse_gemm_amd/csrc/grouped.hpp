// Ragged grouped products: the rows of each expert times that expert's
// weights, with as many rows in a group as the routing left there (no bins
// padded to 128 rows), and the gradient of those weights.
//
//   grouped_gemm    C[r][n] = epilogue(sum_k A[r][k] B_e[k][n]) for the rows r
//                   of expert e, row_offsets[e] <= r < row_offsets[e + 1]
//   grouped_wgrad   C_e[k][n] = sum over those rows r of A[r][k] D[r][n]
//
// One tile body serves them all.  A workgroup of four waves computes an output
// tile of 256 x 256 as four 128 x 128 quadrants of 4 x 4
// v_mfma_f32_32x32x16_bf16 accumulators (v_mfma_f32_32x32x2_f32 for fp32,
// v_mfma_f32_32x32x64_f8f6f4 for e4m3), a group's last rows, when at most 128,
// as a tile of half the height; or tiles of 128 x 256 or 128 x 128, two
// workgroups a compute unit (grouped_plan.cpp says which and why).
//
// Measured, us: dense 8192^3, one expert, bf16 823 (1336 TFLOP/s), e4m3 424
// (2596); e4m3 SwiGLU prompt, 8 experts of 2048 rows, K 4096, N 14336, 1684
// (2290 TFLOP/s); one token of two such experts in bf16 84 (5.6 TB/s of
// weights); 64 experts of 256 rows, K 512, N 2048, GeLU with its derivative,
// 64; weight gradients, 8 experts of 2048 rows, 4096 x 14336, 1600 (1200
// TFLOP/s).  The long loops are bound by the direct loads' address unit (busy
// 96 % of the cycles with both operands K-contiguous, where a row piece is 64
// bytes) and by the power that the matrix cores may draw, the e4m3 products
// also by their epilogues, the few-row products by HBM.
//
// Operand panels of 128 rows x 64 bytes of K go from memory to LDS with
// buffer_load_dwordx4 ... lds through a ring of stages.  The buffer
// descriptor of each operand ends where its data ends: rows past the group,
// columns past the matrix and the K positions behind the last one are out of
// the descriptor's range, which the hardware reads as zero.  So no load of
// another expert's rows reaches an accumulator that is stored, no padding is
// needed in memory, and no address outside the operands is ever read.  (With
// K contiguous, the chunks behind K of the last K-tile lie inside the next
// row; there the lane's offset is set out of range instead.)
//
// The tile list is not built anywhere: the offsets are on the device, the
// launch covers the largest number of tiles that M rows in E groups can
// need, and each workgroup finds its tile by a wave scan over the groups'
// tile counts.
#pragma once

#include <type_traits>

#include "gemm.hpp"

namespace bsg {

template <int DT>
struct GElt;  // K of one 64-byte stage row
template <>
struct GElt<kBf16> {
    static constexpr int kBytes = 2, kKt = 32;
};
template <>
struct GElt<kF32> {
    static constexpr int kBytes = 4, kKt = 16;
};
template <>
struct GElt<kE4m3> {
    static constexpr int kBytes = 1, kKt = 64;
};

// --------------------------------------------------------------- groups

struct Group {
    int e, row0, rows;  // expert, its first row, its rows
    int local;          // tile inside the group's tiles
};

// First row and rows of expert e, kept inside [0, M) whatever the offsets hold.
__device__ __forceinline__ void group_rows(const int32_t* __restrict__ off, int e, int64_t M,
                                           int& row0, int& rows) {
    const int lo = min(max(off[e], 0), (int)M), hi = min(max(off[e + 1], 0), (int)M);
    row0 = lo;
    rows = max(hi - lo, 0);
}

// Inclusive sum over the lanes: within rows of 16 lanes, then across them
// (data-parallel moves: a shuffle through LDS would cost more than the rest
// of the tile search).
__device__ __forceinline__ int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);  // row_shr 1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);  // lane 15 to rows 1, 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);  // lane 31 to rows 2, 3
    return v;
}

// The groups as a wave sees them, 64 at a time: lane l holds expert base + l.
// The first 64 stay in registers between the count and the search.
template <int H>
struct Groups {
    const int32_t* off;
    int E;
    int64_t M;
    int base, row0, rows, incl;  // incl: row tiles of H rows up to and with this expert's

    __device__ __forceinline__ void load(int b, int before) {
        const int e = b + (threadIdx.x & (kWave - 1));
        base = b;
        row0 = rows = 0;
        if (e < E) group_rows(off, e, M, row0, rows);
        incl = wave_scan((rows + H - 1) / H) + before;
    }
    __device__ __forceinline__ int last() const { return __builtin_amdgcn_readlane(incl, kWave - 1); }
    // Row tiles of all groups; leaves the last 64 loaded.
    __device__ __forceinline__ int count() {
        load(0, 0);
        for (int b = kWave; b < E; b += kWave) load(b, last());
        return last();
    }
    // The group of tile `tile` when every row tile has `per` tiles; tile is
    // below count() * per.
    __device__ __forceinline__ Group find(int tile, int per) {
        const int want = tile / per;  // row tile in the order of the groups
        if (base != 0) load(0, 0);
        uint64_t past = __ballot(incl > want);
        while (past == 0 && base + kWave < E) {
            load(base + kWave, last());
            past = __ballot(incl > want);
        }
        const int at = past ? __ffsll((unsigned long long)past) - 1 : 0;
        Group g;
        g.e = base + at;
        g.row0 = __builtin_amdgcn_readlane(row0, at);
        g.rows = __builtin_amdgcn_readlane(rows, at);
        g.local = tile - (__builtin_amdgcn_readlane(incl, at) - (g.rows + H - 1) / H) * per;
        return g;
    }
};

// -------------------------------------------------------------- operands

// One operand of a tile in memory: 256 rows (or columns) as two panels of
// 128, K-tile after K-tile.  `left` bytes from `base` to the end of its data.
struct Operand {
    const char* base;
    int64_t left;
};

// K contiguous: rows [first, first + rows) (256 at most are read) of K_b bytes.
__device__ __forceinline__ Operand operand_k(const void* p, int64_t first, int64_t ld_b, int64_t rows,
                                             int64_t K_b) {
    rows = rows < 256 ? rows : 256;
    return Operand{(const char*)p + first * ld_b, (rows - 1) * ld_b + K_b};
}

// M or N contiguous: k rows of `width_b` bytes, from column byte `col_b` on.
__device__ __forceinline__ Operand operand_n(const void* p, int64_t ld_b, int64_t col_b,
                                             int64_t width_b, int64_t k) {
    return Operand{(const char*)p + col_b, (k - 1) * ld_b + width_b - col_b};
}

// The buffer descriptor of `left` bytes from `base`: raw, offsets in bytes.
// The lane offsets stay below 2^31 (checked on the host), so a range capped
// there cuts nothing off and bit 31 puts a lane out of range.
__device__ __forceinline__ u32x4 descriptor(const char* base, int64_t left) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)left);
    const int hi = __builtin_amdgcn_readfirstlane((int)(left >> 32));
    u32x4 d;
    d[0] = __builtin_amdgcn_readfirstlane((uint32_t)(uint64_t)base);
    d[1] = __builtin_amdgcn_readfirstlane((uint32_t)((uint64_t)base >> 32) & 0xffffu);
    d[2] = hi < 0 ? 0u : hi > 0 || lo > 0x7fffffffu ? 0x7fffffffu : lo;
    d[3] = 0x00020000u;
    return d;
}

// 16 bytes a lane from memory to LDS byte lds_addr + OFF + 16 lane; zeros for
// lanes out of the descriptor's range.  Inline asm for the reason given at
// dma16: the kernel itself waits for these loads before the barrier that
// publishes their stage.  NOP: a vector instruction may have written the
// descriptor's registers just before, which takes five wait states (four here
// after the scalar add; the steps of the main loop set a descriptor a
// barrier or several MFMAs ahead of its next load and need the one of m0 only).
template <int OFF, bool NOP>
__device__ __forceinline__ void dma16_range(uint32_t lds_addr, u32x4 desc, uint32_t off, uint32_t soff) {
    if constexpr (NOP)
        asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 3\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                     :
                     : "s"(lds_addr), "v"(off), "s"(desc), "s"(soff), "n"(OFF)
                     : "memory", "scc");
    else
        asm volatile("s_add_u32 m0, %0, %4\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                     :
                     : "s"(lds_addr), "v"(off), "s"(desc), "s"(soff), "n"(OFF)
                     : "memory", "scc");
}

// Wait until at most N of this wave's loads are in flight (they retire in
// issue order).
template <int N>
__device__ __forceinline__ void wait_loads() {
    static_assert(N >= 0 && N < 64, "the counter's range");
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

typedef int i32x8 __attribute__((ext_vector_type(8)));

// e4m3: both 16-byte K pieces of a stage row at once.  Lane half h holds
// pieces h and 2 + h of the row, for both operands alike, so every k meets
// itself.
__device__ __forceinline__ void mma_e4m3(f32x16& acc, const u32x4* x, const u32x4* y) {
    i32x8 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        a[i] = (int)x[0][i], a[4 + i] = (int)x[1][i];
        b[i] = (int)y[0][i], b[4 + i] = (int)y[1][i];
    }
    // no block scales (zero operands select the plain instruction).  It adds
    // the products of 8 neighbouring k with 13 bits below the largest one
    // (measured: next to a product of 1, products of 2^-13 count and of 2^-14
    // do not), then goes on in fp32.  The rate is twice bf16's, and 7 * 2^-13
    // of the sum of sizes is far below what rounding the operands to e4m3 cost.
    acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc, 0, 0, 0, 0, 0, 0);
}

// f(0), ..., f(N - 1) with the index as a constant.
template <int N, typename F, int I = 0>
__device__ __forceinline__ void unroll(F&& f) {
    if constexpr (I < N) {
        f(std::integral_constant<int, I>{});
        unroll<N, F, I + 1>(static_cast<F&&>(f));
    }
}

// --------------------------------------------------------------- the tile

// Four values of the epilogue: v (and u, the second product) become the
// output, x and y what goes beside it (saved factors; SILU_MUL_BWD: the
// second plane); d and q are the saved factors read.
template <int EPI>
__device__ __forceinline__ void epilogue4(float* v, const float* u, float* x, float* y, const float* d,
                                          const float* q) {
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        if constexpr (EPI == kEpiGelu) {
            v[s] = gelu_f(v[s]);
        } else if constexpr (EPI == kEpiGeluSave) {
            gelu_and_grad(v[s], v[s], x[s]);
        } else if constexpr (EPI == kEpiSiluMul) {
            v[s] = silu_f(v[s]) * u[s];
        } else if constexpr (EPI == kEpiSiluMulSave) {
            float sp;
            silu_and_grad(v[s], x[s], sp);
            y[s] = u[s] * sp;
            v[s] = x[s] * u[s];
        } else if constexpr (EPI == kEpiGeluBwd) {
            v[s] *= d[s];
        } else if constexpr (EPI == kEpiSiluMulBwd) {
            x[s] = v[s] * d[s];
            v[s] *= q[s];
        }
    }
}

__device__ __forceinline__ void unpack4(u32x2 u, float* f) {  // four bf16
    f[0] = __uint_as_float(u[0] << 16);
    f[1] = __uint_as_float(u[0] & 0xffff0000u);
    f[2] = __uint_as_float(u[1] << 16);
    f[3] = __uint_as_float(u[1] & 0xffff0000u);
}

// Whether the epilogue has a second and a third output.
template <int EPI>
constexpr bool kHasX = EPI == kEpiGeluSave || EPI == kEpiSiluMulSave || EPI == kEpiSiluMulBwd;
template <int EPI>
constexpr bool kHasY = EPI == kEpiSiluMulSave;

// What a tile stores: rows [0, mr) x columns [n0, min(N, n0 + width)) of an
// output whose row 0 is the tile's first row.
struct TileOut {
    char* out;            // (tile row 0, column 0)
    char* out2;           // SILU_MUL_BWD: the second plane
    const char* aux_in;   // the saved factors (two planes: aux_in, aux_in2)
    const char* aux_in2;
    char* aux_out;        // the factors to save (two planes: aux_out, aux_out2)
    char* aux_out2;
    const float* a_scale;  // of tile row 0, or NULL
    const float* b_scale;  // of column 0 of the group's weights
    const float* b2_scale;
    float* part;   // SPLIT: a K segment's sums (row 0, column 0; leading dimension N)
    float* part2;  // and, DUAL, those of b2
    int64_t ldc;
    int mr, n0, N;
};

// AK, BK: operand K-contiguous.  PA, PB: panels of A and of B, 1 or 2: the
// tile is 128 PA rows x 128 PB columns, two by two waves of 64 PA x 64 PB
// (DUAL: PB = 2, one panel of each product's B, the tile 128 columns wide).  K
// of one set; sets 2: a second pair of operands into the same accumulators.
// op: A, B (DUAL: its second panel's B) of the first set, then of the second.
// STAGES K-tiles in the ring, of 8 KB a panel.  SPLIT: the sums of a K segment
// go to o.part instead of the epilogue.
template <int DT, bool AK, bool BK, int EPI, int OUT, int PA, int PB, int STAGES, bool SPLIT>
__device__ __forceinline__ void ragged_tile(char* smem, const Operand (*op)[3], int64_t lda_b,
                                             int64_t ldb_b, int64_t K, int sets, const TileOut& o) {
    constexpr int ES = GElt<DT>::kBytes, KT = GElt<DT>::kKt;
    constexpr bool DUAL = EPI == kEpiSiluMul || EPI == kEpiSiluMulSave;
    constexpr int LPT = kSegsPerWave * (PA + PB);  // direct loads per wave and K-tile
    constexpr int NMI = 2 * PA, NNI = 2 * PB;      // 32 x 32 accumulators of a wave
    constexpr int NI = DUAL ? 2 : NNI;             // those of one product, along N
    constexpr int STAGE_BYTES = (PA + PB) * kPanelBytes;
    static_assert(!DUAL || PB == 2, "a panel for each product");
    static_assert(DT != kE4m3 || (AK && BK), "e4m3 operands are K-contiguous");
    lds_t* lds = (lds_t*)smem;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave & 1, wn = wave >> 1, l32 = lane & 31, lh = lane >> 5;
    // the layouts follow the operand's bytes: e4m3 is K-contiguous, where the
    // type does not matter
    constexpr int LT = DT == kE4m3 ? kBf16 : DT;

    const int nk1 = (int)((K + KT - 1) / KT), nk = nk1 * sets;

    // ---- loads: K-tile `lt` is next to go out.  A's panels, then B's.  The
    // second panel of an operand is the first one's descriptor with
    // larger lane offsets.  K-contiguous operands advance through the scalar
    // offset under a constant descriptor; the others move their base.
    constexpr int NOP = DUAL ? 3 : 2;
    uint32_t off[4][kSegsPerWave];
#pragma unroll
    for (int j = 0; j < kSegsPerWave; ++j) {
        const int s = wave * kSegsPerWave + j;
        const uint32_t fa = (uint32_t)seg_offset<LT, AK>(s, lane, lda_b);
        const uint32_t fb = (uint32_t)seg_offset<LT, BK>(s, lane, ldb_b);
        off[0][j] = fa;
        off[1][j] = fa + (uint32_t)(AK ? 128 * lda_b : 128 * ES);
        off[2][j] = fb;
        off[3][j] = DUAL ? fb : fb + (uint32_t)(BK ? 128 * ldb_b : 128 * ES);
    }
    // lanes whose 16 bytes lie behind K in a set's last K-tile (K contiguous;
    // the chunk a lane fetches does not depend on its segment)
    const int last_b = (int)(K - (int64_t)(nk1 - 1) * KT) * ES;
    const uint32_t behind = ((lane & 3) ^ ((lane >> 4) & 3)) * 16 >= last_b ? 0x80000000u : 0u;
    constexpr bool TWO = EPI == kEpiNone;  // may take a second set
    const char* base[NOP];
    int64_t left[NOP];
    u32x4 desc[NOP], desc2[NOP];
#pragma unroll
    for (int i = 0; i < NOP; ++i) {
        base[i] = op[0][i].base;
        left[i] = op[0][i].left;
        desc[i] = descriptor(base[i], left[i]);
        desc2[i] = descriptor(op[1][i].base, op[1][i].left);
    }
    int lt = 0;
    uint32_t soff = 0;                        // bytes of K behind the K-contiguous operands
    uint32_t tail = nk1 == 1 ? behind : 0u;   // `behind` while K-tile lt is a set's last
    const uint32_t lds0 = lds_u32(lds) + wave * kSegsPerWave * 1024;
    uint32_t lds_lt = lds0;                   // this wave's segments in K-tile lt's stage
    // load j (0 .. LPT - 1); FAST: not a set's last K-tile
    auto dma = [&](auto jc, auto fast) {
        constexpr int j = decltype(jc)::value, pnl = j % (PA + PB), sg = j / (PA + PB);
        constexpr int lane_off = pnl < PA ? pnl : 2 + pnl - PA;
        constexpr int i = pnl < PA ? 0 : DUAL && pnl == PA + 1 ? 2 : 1;
        constexpr bool KC = i == 0 ? AK : BK, TAIL = KC && !decltype(fast)::value;
        dma16_range<pnl * kPanelBytes + sg * 1024, !decltype(fast)::value>(
            lds_lt, desc[i], TAIL ? off[lane_off][sg] | tail : off[lane_off][sg], KC ? soff : 0u);
    };
    auto next_stage = [&]() {
        ++lt;
        lds_lt += STAGE_BYTES;
        if (lds_lt == lds0 + STAGES * STAGE_BYTES) lds_lt = lds0;
    };
    // Operands [I0, I1) that move their base: one K-tile on.
    auto advance = [&](int i0, int i1) {
#pragma unroll
        for (int i = i0; i < i1; ++i) {
            if (i == 0 ? AK : BK) continue;
            const int64_t step = KT * (i == 0 ? lda_b : ldb_b);
            base[i] += step;
            left[i] -= step;
            desc[i] = descriptor(base[i], left[i]);
        }
    };
    // One K-tile on, over the end of a set too.  Selects, not branches: behind
    // a branch the compiler gathers the MFMAs that should run among the loads.
    auto next = [&]() {
        next_stage();
        const bool over = lt >= nk, swap = TWO && lt == nk1;
        soff = over || swap ? 0u : soff + kRowBytes;
        tail = lt == nk1 - 1 || lt == nk - 1 ? behind : 0u;
#pragma unroll
        for (int i = 0; i < NOP; ++i) {
            if (i == 0 ? AK : BK) {
                if constexpr (TWO) {
                    desc[i][0] = swap ? desc2[i][0] : desc[i][0];
                    desc[i][1] = swap ? desc2[i][1] : desc[i][1];
                    desc[i][2] = swap ? desc2[i][2] : desc[i][2];
                }
                desc[i][2] = over ? 0u : desc[i][2];
            } else {
                const int64_t step = KT * (i == 0 ? lda_b : ldb_b);
                base[i] = swap ? op[1][i].base : base[i] + step;
                left[i] = swap ? op[1][i].left : left[i] - step;
                desc[i] = descriptor(base[i], over ? 0 : left[i]);
            }
        }
    };

    f32x16 acc[NMI][NNI];
#pragma unroll
    for (int i = 0; i < NMI; ++i)
#pragma unroll
        for (int j = 0; j < NNI; ++j)
#pragma unroll
            for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

    // fragment f (0..NMI-1: A, then B's), K piece c of the K-tile in stage st
    auto read1 = [&](const lds_t* st, int c, int f, u32x4 (*af)[2], u32x4 (*bf)[2]) {
        if (f < NMI) {
            af[f][c] = PA == 1 ? frag<LT, AK>(st, 64 * wm + 32 * f, c)
                               : frag<LT, AK>(st + wm * kPanelBytes, 32 * f, c);
        } else {
            const int ni = f - NMI;
            const int pnl = PA + (DUAL ? ni >> 1 : PB == 1 ? 0 : wn);
            const int row = DUAL ? wn * 64 + 32 * (ni & 1) : PB == 1 ? wn * 64 + 32 * ni : 32 * ni;
            bf[ni][c] = frag<LT, BK>(st + pnl * kPanelBytes, row, c);
        }
    };
    u32x4 af[2][NMI][2], bf[2][NNI][2];
    int rd = 0;  // byte of the stage that the next step reads
    // One K-tile: its MFMAs, and among them the fragment reads of the next
    // one (published by the barrier before) and the loads STAGES ahead into
    // the stage that this K-tile's fragments have left.  Behind the last
    // K-tile the loads are out of range and bring zeros: one wait count
    // throughout, and an odd number of K-tiles ends with one of zeros.  FAST
    // steps, nearly all, stay inside a set and spend few scalar instructions,
    // which would otherwise hold up the next MFMA.
    auto step = [&](auto cur, auto fast) {
        constexpr int c0 = decltype(cur)::value, c1 = 1 - c0;
        constexpr bool FAST = decltype(fast)::value;
        // fragment reads, MFMA groups, and the groups the reads are spread over:
        // the last ones have no reads, so the next barrier finds them returned
        constexpr int NR = 2 * (NMI + NNI), GROUPS = NMI * NNI, READ = GROUPS / 2;
        // the group behind the last load of A (its second segments go out first)
        constexpr int A_OUT = ((PA + PB + PA) * GROUPS - 1) / LPT;
        wait_loads<(STAGES - 2) * LPT>();
        __syncthreads();
        rd += STAGE_BYTES;
        if (rd == STAGES * STAGE_BYTES) rd = 0;
        unroll<GROUPS>([&](auto gc) {
            constexpr int g = decltype(gc)::value;
#pragma unroll
            for (int r = g * NR / READ; r < (g + 1) * NR / READ && r < NR; ++r)
                read1(lds + rd, r & 1, r >> 1, af[c1], bf[c1]);
            constexpr int mi = g / NNI, ni = g % NNI;
            if constexpr (DT != kE4m3) {
                mma<DT>(acc[mi][ni], bf[c0][ni][0], af[c0][mi][0]);
                __builtin_amdgcn_sched_barrier(0);
            }
            constexpr int j0 = g * LPT / GROUPS, j1 = (g + 1) * LPT / GROUPS;
            unroll<j1 - j0>([&](auto jc) {
                dma(std::integral_constant<int, j0 + decltype(jc)::value>{}, fast);
            });
            if constexpr (FAST) {
                if constexpr (g == A_OUT) advance(0, 1);
                if constexpr (g == GROUPS - 1) {
                    advance(1, NOP);
                    soff += kRowBytes;
                    next_stage();
                }
            } else {
                if constexpr (g == GROUPS - 1) next();
            }
            if constexpr (DT == kE4m3) mma_e4m3(acc[mi][ni], bf[c0][ni], af[c0][mi]);
            else mma<DT>(acc[mi][ni], bf[c0][ni][1], af[c0][mi][1]);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    if (nk > 0) {
        using No = std::false_type;
        using Yes = std::true_type;
        for (int t = 0; t < STAGES; ++t) {
            unroll<LPT>([&](auto jc) { dma(jc, No{}); });
            next();
        }
        wait_loads<(STAGES - 1) * LPT>();
        __syncthreads();
#pragma unroll
        for (int f = 0; f < NMI + NNI; ++f) {
            read1(lds, 0, f, af[0], bf[0]);
            read1(lds, 1, f, af[0], bf[0]);
        }
        for (int kt = 0; kt < nk; kt += 2) {
            // steps whose load and the one after it are not the end of a set
            const int fast = (lt < nk1 ? nk1 : nk) - 2 - lt;
            for (int i = fast; i > 1; i -= 2, kt += 2) {
                step(std::integral_constant<int, 0>{}, Yes{});
                step(std::integral_constant<int, 1>{}, Yes{});
            }
            step(std::integral_constant<int, 0>{}, No{});
            step(std::integral_constant<int, 1>{}, No{});
        }
        wait_loads<0>();  // the last (empty) loads still write their stages
    }

    const int wcol = o.n0 + wn * 32 * NI;  // the wave's first column

    // ---- a K segment: fp32 sums as they are, for the launch that adds them
    if constexpr (SPLIT) {
#pragma unroll
        for (int mi = 0; mi < NMI; ++mi) {
            const int row = 64 * PA * wm + 32 * mi + l32;
#pragma unroll
            for (int ni = 0; ni < NNI; ++ni)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int col = wcol + 32 * (DUAL ? ni & 1 : ni) + 8 * g + 4 * lh;
                    float* to = DUAL && ni >= 2 ? o.part2 : o.part;
                    if (row < o.mr && col < o.N)
                        *(f32x4*)(to + (int64_t)row * o.N + col) =
                            f32x4{acc[mi][ni][4 * g], acc[mi][ni][4 * g + 1], acc[mi][ni][4 * g + 2],
                                  acc[mi][ni][4 * g + 3]};
                }
        }
        return;
    }

    // ---- epilogue: bf16 results go through LDS, 32 rows at a time, so that
    // stores write whole rows of 256 (a wave of 64 columns: 128) bytes; fp32 results are
    // stored from the accumulators.  Chunk c of staged row r lies at slot
    // c ^ (r & MASK), which spreads both the writes and the reads over all
    // banks.
    constexpr bool STAGE = OUT == kBf16;
    constexpr int OES = OUT == kBf16 ? 2 : 4;
    constexpr int ROWB = 64 * NI;  // bytes of a staged row
    constexpr int MASK = ROWB / 16 - 1;
    if constexpr (STAGE) __syncthreads();  // the operand ring is free
    static_assert(4 * (DUAL ? 3 : 2) * 32 * ROWB <= STAGES * STAGE_BYTES, "staging fits the ring");
    lds_t* region = lds + wave * ((DUAL ? 3 : 2) * 32 * ROWB);
    if (wcol >= o.N) return;
    auto put = [&](int sub, int chunk, const float* v) {  // row l32
        *(__attribute__((address_space(3))) u32x2*)(region + sub * 32 * ROWB + l32 * ROWB +
                                                      ((chunk ^ (l32 & MASK)) << 4) + lh * 8) =
            u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    };
    auto flush = [&](int sub, char* base, int trow) {
        constexpr int CH = ROWB / 16, RPI = kWave / CH;  // rows an instruction
        const int chunk = lane % CH;
        const int col = wcol + chunk * 8;
#pragma unroll
        for (int rr = 0; rr < 32 / RPI; ++rr) {
            const int row = RPI * rr + lane / CH;
            const u32x4 u = *(const __attribute__((address_space(3))) u32x4*)(
                region + sub * 32 * ROWB + row * ROWB + ((chunk ^ (row & MASK)) << 4));
            if (trow + row < o.mr && col < o.N)
                __builtin_nontemporal_store(u, (u32x4*)(base + ((int64_t)(trow + row) * o.ldc + col) * 2));
        }
    };
    // e4m3: the scales of this lane's rows and columns, all loads in flight at once
    float sa[DT == kE4m3 ? NMI : 1];
    f32x4 sb[DT == kE4m3 ? NI : 1][4], sb2[DT == kE4m3 && DUAL ? NI : 1][4];
    if constexpr (DT == kE4m3) {
#pragma unroll
        for (int mi = 0; mi < NMI; ++mi) {
            const int row = 64 * PA * wm + 32 * mi + l32;
            sa[mi] = row < o.mr ? o.a_scale[row] : 0.0f;
        }
#pragma unroll
        for (int ni = 0; ni < NI; ++ni)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int col = wcol + 32 * ni + 8 * g + 4 * lh;
                const f32x4 zero{0, 0, 0, 0};
                sb[ni][g] = col < o.N ? *(const f32x4*)(o.b_scale + col) : zero;
                if constexpr (DUAL) sb2[ni][g] = col < o.N ? *(const f32x4*)(o.b2_scale + col) : zero;
            }
    }
    constexpr bool ONE_IN = EPI == kEpiGeluBwd || EPI == kEpiSiluMulBwd, TWO_IN = EPI == kEpiSiluMulBwd;
    constexpr bool SLAB_IN = ONE_IN && STAGE;  // bf16: a slab's saved factors are read ahead of it
#pragma unroll
    for (int mi = 0; mi < NMI; ++mi) {
        const int trow = 64 * PA * wm + 32 * mi;  // the slab's first row in the tile
        if (trow >= o.mr) break;
        const int row = trow + l32;
        const bool rin = row < o.mr;
        u32x2 in1[SLAB_IN ? NI : 1][4], in2[SLAB_IN && TWO_IN ? NI : 1][4];
        if constexpr (SLAB_IN) {
#pragma unroll
            for (int ni = 0; ni < NI; ++ni)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const int col = wcol + 32 * ni + 8 * g + 4 * lh;
                    const int64_t at = ((int64_t)row * o.ldc + col) * 2;
                    const bool in = rin && col < o.N;
                    in1[ni][g] = in ? *(const u32x2*)(o.aux_in + at) : u32x2{0, 0};
                    if constexpr (TWO_IN) in2[ni][g] = in ? *(const u32x2*)(o.aux_in2 + at) : u32x2{0, 0};
                }
        }
#pragma unroll
        for (int ni = 0; ni < NI; ++ni) {
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int col = wcol + 32 * ni + 8 * g + 4 * lh;
                const bool in = rin && col < o.N;
                const int64_t at = ((int64_t)row * o.ldc + col) * OES;
                float v[4], u[4];
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    v[s] = acc[mi][ni][4 * g + s];
                    if constexpr (DUAL) u[s] = acc[mi][ni + 2][4 * g + s];
                    if constexpr (DT == kE4m3) {
                        v[s] *= sa[mi] * sb[ni][g][s];
                        if constexpr (DUAL) u[s] *= sa[mi] * sb2[ni][g][s];
                    }
                }
                float x[4], y[4], d[4] = {0, 0, 0, 0}, q[4] = {0, 0, 0, 0};
                if constexpr (SLAB_IN) {
                    unpack4(in1[ni][g], d);
                    if constexpr (TWO_IN) unpack4(in2[ni][g], q);
                } else if constexpr (ONE_IN) {
                    if (in) load4<OUT>(o.aux_in + at, d);
                    if constexpr (TWO_IN) {
                        if (in) load4<OUT>(o.aux_in2 + at, q);
                    }
                }
                epilogue4<EPI>(v, u, x, y, d, q);
                constexpr bool X = kHasX<EPI>, Y = kHasY<EPI>;
                if constexpr (STAGE) {
                    put(0, 4 * ni + g, v);
                    if constexpr (X) put(1, 4 * ni + g, x);
                    if constexpr (Y) put(2, 4 * ni + g, y);
                } else if (in) {
                    store4<OUT>(o.out + at, v);
                    if constexpr (X) store4<OUT>((EPI == kEpiSiluMulBwd ? o.out2 : o.aux_out) + at, x);
                    if constexpr (Y) store4<OUT>(o.aux_out2 + at, y);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (STAGE) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            flush(0, o.out, trow);
            if constexpr (EPI == kEpiGeluSave || EPI == kEpiSiluMulSave) flush(1, o.aux_out, trow);
            if constexpr (EPI == kEpiSiluMulBwd) flush(1, o.out2, trow);
            if constexpr (EPI == kEpiSiluMulSave) flush(2, o.aux_out2, trow);
        }
    }
}

// ----------------------------------------------------------------- kernels

// Row tiles of one group taken together, down the rows first (see
// grouped_tile in common.hpp), and kGroupedChunk consecutive tiles, one for
// each compute unit of an XCD, dealt to the XCDs in turn: what an XCD runs at
// once is 4 x 8 tiles that share both operands' panels in its L2, and the chip
// works on one region of the output.  Against a contiguous eighth of all tiles
// for each XCD, with 8 rows together, us: 8 experts of 2048 rows, K 14336,
// N 4096: 1827 -> 1661; e4m3 SwiGLU, K 4096, N 14336: 1752 -> 1684; 64 skewed
// experts, K 4096, N 1024: 1085 -> 1041; K 1024, N 4096: 1214 -> 1248.  Groups
// of a few rows read each weight once in either order, and fastest from
// contiguous ranges: 8 experts of 12 rows, K 4096, e4m3 196 against 203.
constexpr int kGroupedRows = 4;
constexpr int kGroupedChunk = 32;
constexpr int kChunkedRows = 64;  // rows a group on average from which chunks are dealt

// H x W: rows and columns of a tile (DUAL: W = 256, of which each product has
// 128).  256 rows: one workgroup a compute unit, a group's last rows (at most
// 128) as a tile of half the height.  128: two workgroups a compute unit, one's
// loads and stores beside the other's products.
template <int H, int W>
struct TileShape {
    static constexpr int kHalfStages = H == 256 ? 5 : W == 256 ? 3 : 4;
    static constexpr int kLds = H == 256 ? kStages * kStageBytes : kHalfStages * (1 + W / 128) * kPanelBytes;
    static constexpr int kPerCu = H == 256 ? 1 : 2;
};

template <int DT, bool BK, int EPI, int OUT, int H, int W, bool SPLIT>
__global__ __launch_bounds__(kGemmThreads, (TileShape<H, W>::kPerCu)) void grouped_gemm_kernel(GroupedParams P) {
    constexpr int ES = GElt<DT>::kBytes, KT = GElt<DT>::kKt;
    constexpr bool DUAL = EPI == kEpiSiluMul || EPI == kEpiSiluMulSave;
    constexpr int OES = OUT == kBf16 ? 2 : 4;
    __shared__ __attribute__((aligned(1024))) char smem[TileShape<H, W>::kLds];
    constexpr int TW = DUAL ? 128 : W;  // columns of the output
    const int tn = (P.N + TW - 1) / TW;
    Groups<H> groups{P.row_offsets, P.E, P.M};
    const int ntiles = groups.count() * tn;
    const int nseg = SPLIT ? P.nseg : 1;
    if ((int)blockIdx.x >= ntiles * nseg) return;
    // split: segment-major, so that what an XCD runs at once shares one K segment
    const bool dealt = !SPLIT && P.M >= (int64_t)kChunkedRows * P.E;
    const int v = dealt ? xcd_chunked(blockIdx.x, ntiles, kGroupedChunk) : xcd_remap(blockIdx.x, ntiles * nseg);
    const int seg = SPLIT ? v / ntiles : 0;
    const Group g = groups.find(v - seg * ntiles, tn);
    // offsets that do not ascend may add up to more tiles than an int holds
    if ((unsigned)g.local >= (unsigned)((g.rows + H - 1) / H * tn)) return;
    int tm, tq;
    grouped_tile(g.local, (g.rows + H - 1) / H, tn, kGroupedRows, tm, tq);
    const int mr = min(H, g.rows - H * tm);
    const int64_t row = (int64_t)g.row0 + H * tm;
    const int n0 = tq * TW;
    int k0 = 0, K = P.K;
    if constexpr (SPLIT) {  // the segment's K
        const int nk = (P.K + KT - 1) / KT;
        k0 = (int)((int64_t)nk * seg / nseg) * KT;
        K = min(P.K, (int)((int64_t)nk * (seg + 1) / nseg) * KT) - k0;
    }
    const int64_t lda_b = P.lda * ES, ldb_b = P.ldb * ES, K_b = (int64_t)K * ES;
    const int64_t eb = (int64_t)g.e * P.stride_b * ES;
    auto B = [&](const void* b) {
        const char* be = (const char*)b + eb + (int64_t)k0 * (BK ? ES : ldb_b);
        if constexpr (BK) return operand_k(be, n0, ldb_b, P.N - n0, K_b);
        else return operand_n(be, ldb_b, (int64_t)n0 * ES, (int64_t)P.N * ES, K);
    };
    auto A = [&](const void* a) { return operand_k((const char*)a + (int64_t)k0 * ES, row, lda_b, mr, K_b); };
    const Operand op[2][3] = {{A(P.a), B(P.b), B(P.b2)}, {A(P.a2), B(P.b2), B(P.b2)}};
    TileOut o{};
    o.ldc = P.ldc;
    o.mr = mr;
    o.n0 = n0;
    o.N = P.N;
    const int64_t at = row * P.ldc * OES, plane = P.M * P.ldc * OES;
    o.out = (char*)P.c + at;
    o.out2 = o.out + plane;
    o.aux_in = (const char*)P.aux_in + at;
    o.aux_in2 = o.aux_in + plane;
    o.aux_out = (char*)P.aux_out + at;
    o.aux_out2 = o.aux_out + plane;
    if constexpr (DT == kE4m3) {
        o.a_scale = P.a_scale + row;
        o.b_scale = P.b_scale + (int64_t)g.e * P.N;
        o.b2_scale = o.b_scale + (int64_t)P.E * P.N;
    }
    if constexpr (SPLIT) {
        const int64_t share = P.M * P.N;
        o.part = P.ws + (int64_t)seg * (DUAL ? 2 : 1) * share + row * P.N;
        o.part2 = o.part + share;
    }
    const int sets = EPI == kEpiNone && P.a2 ? 2 : 1;
    if constexpr (H == 256) {
        if (mr > 128) {
            ragged_tile<DT, true, BK, EPI, OUT, 2, W / 128, kStages, SPLIT>(smem, op, lda_b, ldb_b, K, sets, o);
            return;
        }
    }
    ragged_tile<DT, true, BK, EPI, OUT, 1, W / 128, TileShape<H, W>::kHalfStages, SPLIT>(
        smem, op, lda_b, ldb_b, K, sets, o);
}

// The second launch of a split product: a workgroup a row and 1024 columns,
// the segments' sums added in order, then scales and epilogue as in the tile.
template <int DT, int EPI, int OUT>
__global__ __launch_bounds__(kGemmThreads) void grouped_join_kernel(GroupedParams P) {
    constexpr bool DUAL = EPI == kEpiSiluMul || EPI == kEpiSiluMulSave;
    constexpr int OES = OUT == kBf16 ? 2 : 4;
    const int64_t row = blockIdx.x;
    const int first = P.row_offsets[0], end = P.row_offsets[P.E];
    if (row < first || row >= end) return;  // a row of no group
    const int col = (blockIdx.y * kGemmThreads + threadIdx.x) * 4;
    if (col >= P.N) return;
    const int64_t share = P.M * P.N;
    const float* part = P.ws + row * P.N + col;
    float v[4] = {0, 0, 0, 0}, u[4] = {0, 0, 0, 0};
#pragma unroll 4
    for (int i = 0; i < P.nseg; ++i) {
        const f32x4 p = *(const f32x4*)(part + (int64_t)i * (DUAL ? 2 : 1) * share);
#pragma unroll
        for (int s = 0; s < 4; ++s) v[s] += p[s];
        if constexpr (DUAL) {
            const f32x4 p2 = *(const f32x4*)(part + (int64_t)(2 * i + 1) * share);
#pragma unroll
            for (int s = 0; s < 4; ++s) u[s] += p2[s];
        }
    }
    if constexpr (DT == kE4m3) {
        int lo = 0, hi = P.E - 1;  // the last expert that starts at or before the row
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (P.row_offsets[mid] <= row) lo = mid;
            else hi = mid - 1;
        }
        const float sa = P.a_scale[row];
        const float* sb = P.b_scale + (int64_t)lo * P.N + col;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            v[s] *= sa * sb[s];
            if constexpr (DUAL) u[s] *= sa * sb[(int64_t)P.E * P.N + s];
        }
    }
    const int64_t at = (row * P.ldc + col) * OES, plane = P.M * P.ldc * OES;
    float x[4], y[4], d[4] = {0, 0, 0, 0}, q[4] = {0, 0, 0, 0};
    if constexpr (EPI == kEpiGeluBwd || EPI == kEpiSiluMulBwd) load4<OUT>((const char*)P.aux_in + at, d);
    if constexpr (EPI == kEpiSiluMulBwd) load4<OUT>((const char*)P.aux_in + plane + at, q);
    epilogue4<EPI>(v, u, x, y, d, q);
    store4<OUT>((char*)P.c + at, v);
    if constexpr (EPI == kEpiSiluMulBwd) store4<OUT>((char*)P.c + plane + at, x);
    else if constexpr (kHasX<EPI>) store4<OUT>((char*)P.aux_out + at, x);
    if constexpr (kHasY<EPI>) store4<OUT>((char*)P.aux_out + plane + at, y);
}

// Weight gradients: C_e [K x N], the reduction along the group's rows; both
// operands are read as they lie, row by row.  Groups in order, a group's
// tiles four high; groups without rows store zeros.
// SPLIT: P.nseg segments of each group's rows, their sums to the workspace.
template <int DT, int OUT, int H, int W, bool SPLIT>
__global__ __launch_bounds__(kGemmThreads, (TileShape<H, W>::kPerCu)) void grouped_wgrad_kernel(GroupedParams P) {
    constexpr int ES = GElt<DT>::kBytes, KT = GElt<DT>::kKt;
    constexpr int OES = OUT == kBf16 ? 2 : 4;
    __shared__ __attribute__((aligned(1024))) char smem[TileShape<H, W>::kLds];
    const int tk = (P.K + H - 1) / H, tn = (P.N + W - 1) / W;
    const int per = tk * tn, ntiles = P.E * per;
    const int seg = SPLIT ? blockIdx.x / ntiles : 0;
    const int t = SPLIT ? (int)blockIdx.x - seg * ntiles : xcd_chunked(blockIdx.x, ntiles, kDstdChunk);
    const int e = t / per;
    int tm, tq;
    grouped_tile(t - e * per, tk, tn, 4, tm, tq);
    int row0, rows;
    group_rows(P.row_offsets, e, P.M, row0, rows);
    row0 = __builtin_amdgcn_readfirstlane(row0);
    rows = __builtin_amdgcn_readfirstlane(rows);
    if constexpr (SPLIT) {  // the segment's rows
        const int nk = (rows + KT - 1) / KT;
        const int k0 = (int)((int64_t)nk * seg / P.nseg) * KT;
        const int k1 = min(rows, (int)((int64_t)nk * (seg + 1) / P.nseg) * KT);
        row0 += k0;
        rows = max(k1 - k0, 0);
    }
    const int64_t lda_b = P.lda * ES, ldb_b = P.ldb * ES;
    const char* A = (const char*)P.a + (int64_t)row0 * lda_b;
    const char* D = (const char*)P.b + (int64_t)row0 * ldb_b;
    const Operand oa = operand_n(A, lda_b, (int64_t)tm * H * ES, (int64_t)P.K * ES, rows);
    const Operand ob = operand_n(D, ldb_b, (int64_t)tq * W * ES, (int64_t)P.N * ES, rows);
    const Operand op[2][3] = {{oa, ob, ob}, {oa, ob, ob}};
    TileOut o{};
    o.ldc = P.ldc;
    o.mr = min(H, P.K - H * tm);
    o.n0 = tq * W;
    o.N = P.N;
    o.out = (char*)P.c + ((int64_t)e * P.stride_b + (int64_t)tm * H * P.ldc) * OES;
    if constexpr (SPLIT) o.part = P.ws + (((int64_t)seg * P.E + e) * P.K + (int64_t)tm * H) * P.N;
    if constexpr (H == 256) {
        if (o.mr > 128) {
            ragged_tile<DT, false, false, kEpiNone, OUT, 2, W / 128, kStages, SPLIT>(smem, op, lda_b, ldb_b,
                                                                                     rows, 1, o);
            return;
        }
    }
    ragged_tile<DT, false, false, kEpiNone, OUT, 1, W / 128, TileShape<H, W>::kHalfStages, SPLIT>(
        smem, op, lda_b, ldb_b, rows, 1, o);
}

// The second launch of a split weight gradient: row k of expert e, the
// segments' sums added in order.
template <int OUT>
__global__ __launch_bounds__(kGemmThreads) void grouped_wgrad_join_kernel(GroupedParams P) {
    constexpr int OES = OUT == kBf16 ? 2 : 4;
    const int64_t row = blockIdx.x;  // e K + k
    const int col = (blockIdx.y * kGemmThreads + threadIdx.x) * 4;
    if (col >= P.N) return;
    const int64_t share = (int64_t)P.E * P.K * P.N;
    float v[4] = {0, 0, 0, 0};
#pragma unroll 4
    for (int i = 0; i < P.nseg; ++i) {
        const f32x4 p = *(const f32x4*)(P.ws + i * share + row * P.N + col);
#pragma unroll
        for (int s = 0; s < 4; ++s) v[s] += p[s];
    }
    const int64_t e = row / P.K, k = row - e * P.K;
    store4<OUT>((char*)P.c + (e * P.stride_b + k * P.ldc + col) * OES, v);
}

// Most tiles of M rows in E groups, `per` tiles a row tile of H rows: every
// group that has rows ends in at most one tile that is not full.
inline int64_t grouped_tiles_max(int64_t M, int E, int H, int64_t per) {
    const int64_t ne = E < M ? E : M;
    return ((M + (int64_t)(H - 1) * ne) / H) * per;
}

template <int DT, bool BK, int EPI, int OUT, int H, int W, bool SPLIT>
static hipError_t grouped_go_tile(const GroupedParams& p, hipStream_t s) {
    constexpr int TW = EPI == kEpiSiluMul || EPI == kEpiSiluMulSave ? 128 : W;
    const int64_t grid = grouped_tiles_max(p.M, p.E, H, (p.N + TW - 1) / TW) * (SPLIT ? p.nseg : 1);
    hipLaunchKernelGGL((grouped_gemm_kernel<DT, BK, EPI, OUT, H, W, SPLIT>), dim3((unsigned)grid),
                       dim3(kGemmThreads), 0, s, p);
    return hipGetLastError();
}

template <int DT, bool BK, int EPI, int OUT>
static hipError_t grouped_go(const GroupedParams& p, hipStream_t s) {
    constexpr bool DUAL = EPI == kEpiSiluMul || EPI == kEpiSiluMulSave;
    if (p.nseg > 1) {  // few rows: the segments' kernel knows no epilogue, the join does
        constexpr int E = DUAL ? kEpiSiluMul : kEpiNone;
        const hipError_t e = p.tile_rows == 128 ? grouped_go_tile<DT, BK, E, kF32, 128, 256, true>(p, s)
                                                : grouped_go_tile<DT, BK, E, kF32, 256, 256, true>(p, s);
        if (e != hipSuccess) return e;
        hipLaunchKernelGGL((grouped_join_kernel<DT, EPI, OUT>),
                           dim3((unsigned)p.M, (unsigned)((p.N + 4 * kGemmThreads - 1) / (4 * kGemmThreads))),
                           dim3(kGemmThreads), 0, s, p);
        return hipGetLastError();
    }
    if constexpr (!DUAL) {
        if (p.tile_cols == 128) return grouped_go_tile<DT, BK, EPI, OUT, 128, 128, false>(p, s);
    }
    return p.tile_rows == 128 ? grouped_go_tile<DT, BK, EPI, OUT, 128, 256, false>(p, s)
                              : grouped_go_tile<DT, BK, EPI, OUT, 256, 256, false>(p, s);
}

}  // namespace bsg
