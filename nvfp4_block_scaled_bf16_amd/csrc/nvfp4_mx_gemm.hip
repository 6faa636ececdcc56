// nvfp4_mx_gemm.hip -- products of MXFP4 operands for gfx950 (format and
// layout: nvfp4_mx.hpp).
//   out[m][n] = sum_k a[m][k] b[n][k],  a and b the values their codes stand for
// dense, by groups of rows with a b of their own each, and summed over each
// group's rows (the groups' weight gradients).  The scaled MFMA multiplies a
// block's 32 codes and both operands' scales in the matrix core and adds in
// fp32; nothing is dequantized on the way.  Each output is rounded once, to
// its type.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "nvfp4_mx.hpp"

namespace nvfp4 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kFp4 = 4;   // the MFMA's format selector for E2M1

// the MFMA's operand registers: an FP4 operand uses the first four
__device__ __forceinline__ i32x8 frag(u32x4 v) { return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0}; }

// two values of a 16-bit output type, the first in the low half
__device__ __forceinline__ uint32_t pack16(int type, float a, float b) {
    if (type == MX_BF16) return bf16x2_rne(a, b);
    const mx_f16x2 h = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, h);
}

// ------------------------------------------------------------ many rows
//
// A workgroup of WM x WN waves computes a BM x BN tile in stages of 256
// elements: 128 code bytes (a whole cache line) and two scale words of every
// operand row, brought to LDS by loads that go there directly, one stage in
// use and one on its way.  A wave keeps (BM / WM) x (BN / WN) of the tile in
// 32 x 32 accumulators; v_mfma_scale 32x32x64 takes row l % 32 of an operand
// in lane l, lanes 0-31 one block and lanes 32-63 another.  Lanes 0-31 take
// blocks 0 .. 3 of the stage and lanes 32-63 blocks 4 .. 7, one of each to a
// quarter, so that a lane's scales for the whole stage are one word.
//
// LDS: row r's eight 16-byte chunks at 128 r, chunk c in place c ^ (r % 8): 8
// lanes reading one chunk of 8 rows touch every bank once.
//
// What bounds it is power: random codes hold the chip near 1.45 GHz (the
// matrix cores alone, without any load, run at 1.6 GHz and reach 6.4 PFLOP/s),
// and the loop takes 1325 cycles per 128 elements where the matrix cores need
// 1024.  16384 x 8192 x 8192: 575 us = 3.8 PFLOP/s.  Steps that led here, same
// size: 128 x 128 tiles, 128-element stages, all of a stage's reads and loads
// before its MFMAs 863 us; 256 x 256 tiles 730; outputs turned around in LDS
// instead of 2-byte stores, tiles in XCD order 691; whole cache lines and each
// LDS read and load placed between MFMAs 575 (the reads alone held up the
// MFMAs for 400 cycles a step, the loads, half a line each, for another 400).

enum GemmMode { GEMM_DENSE, GEMM_GROUPED, GEMM_WGRAD };

template <int BM, int BN>
struct GemmStage {
    uint8_t q[(BM + BN) * 128];
    uint32_t sf[2][BM + BN];
};

typedef const __attribute__((address_space(1))) uint32_t* GlobalPtr;
typedef __attribute__((address_space(3))) uint32_t* LdsPtr;

// each lane's bytes to dst + 16 (4) * lane
__device__ __forceinline__ void load16_to_lds(const uint8_t* src, void* dst) {
    __builtin_amdgcn_global_load_lds((GlobalPtr)src, (LdsPtr)dst, 16, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(const uint8_t* src, void* dst) {
    __builtin_amdgcn_global_load_lds((GlobalPtr)src, (LdsPtr)dst, 4, 0, 0);
}

// The workgroups of a launch go to the 8 XCDs in turn; each XCD takes a
// contiguous run of tiles, so that its L2 holds the operand rows they share.
__device__ __forceinline__ uint32_t xcd_index() {
    const uint32_t g = gridDim.x, x = blockIdx.x & 7u, i = blockIdx.x >> 3;
    return x * (g >> 3) + (x < (g & 7u) ? x : (g & 7u)) + i;
}

// Tile t of ntm x ntn in bands of kBand rows of tiles, down a band's tiles of
// one column and then the next: the 32 tiles that an XCD works on at a time
// share 8 tiles of a and 4 of b.
constexpr uint32_t kBand = 8;
__device__ __forceinline__ void band_tile(uint32_t t, uint32_t ntm, uint32_t ntn, uint32_t* tm, uint32_t* tn) {
    const uint32_t per = kBand * ntn, g = t / per, first = g * kBand;
    const uint32_t gm = ntm - first < kBand ? ntm - first : kBand, w = t - g * per;
    *tm = first + w % gm;
    *tn = w / gm;
}

struct TileArgs {
    const uint8_t *a_q, *a_sf, *b_q, *b_sf;
    int64_t A, M, N, Kt;             // rows of a, rows and columns of out (per group in GEMM_WGRAD), steps of a row
    void* out;
    int type;
    const int32_t* offsets;
    int E;
    int64_t R;
    const int32_t* rows;
    const float* row_scale;
    uint32_t ntm, ntn;
};

// bytes in which a wave turns 32 rows of its output around: 128 16-bit or 64
// fp32 values each, and 16 bytes that keep the rows' banks apart
constexpr int kSlab = 32 * (256 + 16);

// Rows [row0, row0 + nrow) and columns [col0, col0 + ncol) of out from a slab
// of W values a row (T: 2- or 4-byte values), by one wave
template <typename T, int W>
__device__ __forceinline__ void store_slab(const T* slab, T* out, int64_t N, int nrow, int ncol, bool wide, int lane) {
    constexpr int P = W + 16 / (int)sizeof(T), V = 16 / (int)sizeof(T), PER = W / V;
    if (wide && ncol >= W) {
#pragma unroll 4
        for (int r = lane / PER; r < nrow; r += 64 / PER)
            *(u32x4*)(out + r * N + V * (lane % PER)) = *(const u32x4*)&slab[r * P + V * (lane % PER)];
    } else {
        for (int r = 0; r < nrow; ++r)
            for (int c = lane; c < W && c < ncol; c += 64) out[r * N + c] = slab[r * P + c];
    }
}

template <int BM, int BN, int WM, int WN, int MODE>
__global__ __launch_bounds__(64 * WM * WN) void k_mx_gemm(TileArgs p) {
    constexpr int NT = 64 * WM * WN, FM = BM / WM / 32, FN = BN / WN / 32;
    // loads a thread issues per stage: of a's codes, b's and the scales
    constexpr int QA = BM * 8 / NT, QB = BN * 8 / NT, SL = 2 * (BM + BN) / NT, L = QA + QB + SL;
    static_assert(BM * 8 % NT == 0 && BN * 8 % NT == 0 && 2 * (BM + BN) % NT == 0 && BM % 64 == 0 && BN % 64 == 0, "");
    static_assert(WM * WN * kSlab <= 2 * (int)sizeof(GemmStage<BM, BN>), "");
    __shared__ __attribute__((aligned(16))) GemmStage<BM, BN> S[2];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN, half = lane >> 5, lr = lane & 31;

    int64_t m0, n0, mend = p.M, step0 = 0, steps = p.Kt, out0 = 0;
    const uint8_t *b_q = p.b_q, *b_sf = p.b_sf;
    {
        uint32_t id = xcd_index(), tm, tn;
        if constexpr (MODE == GEMM_WGRAD) {
            const uint32_t per = p.ntm * p.ntn;
            const int e = (int)(id / per);
            id -= (uint32_t)e * per;
            // the group's steps in the padded rows follow those of the groups before it
            int before = 0;
            for (int e0 = 0; e0 < e; e0 += 64) {
                int64_t a = 0, b = 0;
                if (e0 + lane < e) mx_group_rows(p.offsets, e0 + lane, p.R, &a, &b);
                int n = (int)((b - a + 127) >> 7);
#pragma unroll
                for (int d = 32; d; d >>= 1) n += __shfl_xor(n, d, 64);
                before += n;
            }
            int64_t a, b;
            mx_group_rows(p.offsets, e, p.R, &a, &b);
            step0 = __builtin_amdgcn_readfirstlane(before);
            steps = (b - a + 127) >> 7;
            // offsets that are not in order could ask for more steps than there are
            if (step0 + steps > p.Kt) steps = p.Kt > step0 ? p.Kt - step0 : 0;
            out0 = (int64_t)e * p.M * p.N;
        }
        if constexpr (MODE == GEMM_GROUPED) {
            tn = id % p.ntn;
            const MxGroupTile g = mx_find_group(p.offsets, p.E, p.R, BM, id / p.ntn);
            if (g.e < 0) return;
            m0 = g.begin;
            mend = g.end;
            b_q += (int64_t)g.e * p.N * p.Kt * 64;
            b_sf += (int64_t)g.e * ((p.N + 127) / 128) * p.Kt * 512;
        } else {
            band_tile(id, p.ntm, p.ntn, &tm, &tn);
            m0 = (int64_t)tm * BM;
        }
        n0 = (int64_t)tn * BN;
    }

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int a = 0; a < 16; ++a) acc[i][j][a] = 0.0f;

    if (steps > 0) {
        // Sources of this thread's loads: row (tid + NT i) / 8 of the tile,
        // chunk qc.  Rows past the end repeat the last one, whose products are
        // not stored.  Grouped rows can be anywhere in a: 64-bit offsets.
        constexpr bool GA = MODE == GEMM_GROUPED;
        typedef typename std::conditional<GA, int64_t, uint32_t>::type AOff;
        const uint8_t* const abase = GA ? p.a_q : p.a_q + (m0 * p.Kt + step0) * 64;
        const uint8_t* const bbase = b_q + (n0 * p.Kt + step0) * 64;
        auto arow = [&](int r) {
            int64_t row = m0 + r < mend ? m0 + r : mend - 1;
            if constexpr (GA) {
                if (p.rows) row = p.rows[row];
                row = row < 0 ? 0 : (row < p.A ? row : p.A - 1);
            }
            return row;
        };
        const int qc = (tid & 7) ^ ((tid >> 3) & 7);
        AOff qa[QA];
        uint32_t qb[QB];
#pragma unroll
        for (int i = 0; i < QA; ++i)
            qa[i] = (AOff)((arow((tid + NT * i) >> 3) - (GA ? 0 : m0)) * (p.Kt * 64) + 16 * qc);
#pragma unroll
        for (int i = 0; i < QB; ++i) {
            const int r = (tid + NT * i) >> 3;
            qb[i] = (uint32_t)(n0 + r < p.N ? r : p.N - 1 - n0) * (uint32_t)(p.Kt * 64) + 16 * qc;
        }
        // scale words: the stage's first step's of all rows, then the second's
        const uint8_t* sp[SL];
        int second[SL];
#pragma unroll
        for (int i = 0; i < SL; ++i) {
            const int first = 64 * wave + NT * i, w = first >= BM + BN, f = first - w * (BM + BN), r = f + lane;
            const int64_t row = f < BM ? arow(r) : (n0 + r - BM < p.N ? n0 + r - BM : p.N - 1);
            sp[i] = (f < BM ? p.a_sf : b_sf) + mx_sf_offset(row, step0, p.Kt);
            second[i] = w ? 512 : 0;
        }
        const int64_t nst = (steps + 1) >> 1, nfull = steps >> 1;
        // an odd last step's stage takes it twice, the second time as zeros
        const uint32_t back = (uint32_t)(qc & 4) * 16;
        auto bring = [&](int n, int64_t k, GemmStage<BM, BN>& st) __attribute__((always_inline)) {
            const bool cut = 2 * k + 1 >= steps;
            const uint32_t bb = cut ? back : 0u;
            if (n < QA) {
                load16_to_lds(abase + k * 128 + (qa[n] - bb), &st.q[16 * (64 * wave + NT * n)]);
            } else if (n < QA + QB) {
                load16_to_lds(bbase + k * 128 + (qb[n - QA] - bb), &st.q[128 * BM + 16 * (64 * wave + NT * (n - QA))]);
            } else {
                const int i = n - QA - QB;
                load4_to_lds(sp[i] + k * 1024 + (cut ? 0 : second[i]), &st.sf[0][64 * wave + NT * i]);
            }
        };

        // operand tiles z: b's, then a's
        struct Frags { u32x4 v[FM + FN]; };
        struct Scales { int v[FM + FN]; };
        auto tile_row = [&](int z) { return z < FN ? BM + wn * (BN / WN) + 32 * z + lr : wm * (BM / WM) + 32 * (z - FN) + lr; };
        auto read = [&](const GemmStage<BM, BN>& st, int quarter, int z, Frags& f) __attribute__((always_inline)) {
            f.v[z] = *(const u32x4*)&st.q[tile_row(z) * 128 + 16 * ((4 * half + quarter) ^ (lr & 7))];
        };
        auto read_scale = [&](const GemmStage<BM, BN>& st, int z, Scales& f) __attribute__((always_inline)) {
            f.v[z] = (int)st.sf[half][tile_row(z)];
        };
        // The products of one quarter of a stage (`use`, `sc`).  Between them,
        // in the order written: the reads of the next quarter (quarter rq of
        // stage rst into `nxt`; its scales where `ns` is given), done by two
        // thirds of the way, and loads l0 .. l1 of stage k into `into`.
        auto quarter = [&](auto Q, const Frags& use, const Scales& sc, Frags& nxt, const GemmStage<BM, BN>& rst, int rq,
                           Scales* ns, int l0, int l1, int64_t k, GemmStage<BM, BN>& into) __attribute__((always_inline)) {
            constexpr int P = FM * FN, Z = FM + FN;
            int z = 0, l = l0;
#pragma unroll
            for (int n = 0; n < P; ++n) {
                const int want = (n + 1) * Z * 3 / (P * 2) + 1, zt = rq < 0 ? 0 : (n + 1 == P || want > Z ? Z : want);
#pragma unroll
                for (int t = 0; t < Z; ++t)
                    if (t >= z && t < zt) {
                        read(rst, rq, t, nxt);
                        if (ns) read_scale(rst, t, *ns);
                    }
                z = zt;
                const int lt = l0 + (l1 - l0) * (n + 1) / P;
#pragma unroll
                for (int t = 0; t < L; ++t)
                    if (t >= l && t < lt) bring(t, k, into);
                l = lt;
                const int i = n / FN, j = n % FN;
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                    frag(use.v[j]), frag(use.v[FN + i]), acc[i][j], kFp4, kFp4, decltype(Q)::value, sc.v[j],
                    decltype(Q)::value, sc.v[FN + i]);
                __builtin_amdgcn_sched_barrier(0);
            }
        };
        using Q0 = std::integral_constant<int, 0>;
        using Q1 = std::integral_constant<int, 1>;
        using Q2 = std::integral_constant<int, 2>;
        using Q3 = std::integral_constant<int, 3>;
        Frags f0, f1;
        Scales sc, sn;
        // A stage's loads begin in the last quarter of the stage two before it,
        // whose place it takes, and end two quarters on
        constexpr int L1 = L / 2;
#pragma unroll
        for (int n = 0; n < L; ++n) bring(n, 0, S[0]);
#pragma unroll
        for (int n = 0; n < L1; ++n) bring(n, nst > 1 ? 1 : 0, S[1]);
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(L1) : "memory");
#pragma unroll
        for (int z = 0; z < FM + FN; ++z) {
            read(S[0], 0, z, f0);
            read_scale(S[0], z, sc);
        }
        auto stage = [&](int64_t s, GemmStage<BM, BN>& cur, GemmStage<BM, BN>& oth) __attribute__((always_inline)) {
            // past the last stage its loads come again, into a place that nobody reads
            const int64_t k1 = s + 1 < nst ? s + 1 : nst - 1, k2 = s + 2 < nst ? s + 2 : nst - 1;
            __builtin_amdgcn_sched_barrier(0);
            quarter(Q0{}, f0, sc, f1, cur, 1, nullptr, L1, L, k1, oth);
            quarter(Q1{}, f1, sc, f0, cur, 2, nullptr, L, L, k1, oth);
            quarter(Q2{}, f0, sc, f1, cur, 3, nullptr, L, L, k1, oth);
            // the next stage has landed, and this one has been read by every wave
            asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
            __builtin_amdgcn_sched_barrier(0);
            quarter(Q3{}, f1, sc, f0, oth, 0, &sn, 0, L1, k2, cur);
            sc = sn;
        };
        for (int64_t s = 0; s < nfull; s += 2) {
            stage(s, S[0], S[1]);
            if (s + 1 < nfull) stage(s + 1, S[1], S[0]);
        }
        if (nst > nfull) {
            auto drop = [&](Frags& f) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < FM; ++i) f.v[FN + i] = half ? u32x4{0, 0, 0, 0} : f.v[FN + i];
            };
#pragma unroll
            for (int z = 0; z < FM + FN; ++z) sc.v[z] = half ? 0 : sc.v[z];
            GemmStage<BM, BN>& cur = S[nfull & 1];
            drop(f0);
            quarter(Q0{}, f0, sc, f1, cur, 1, nullptr, L, L, 0, cur);
            drop(f1);
            quarter(Q1{}, f1, sc, f0, cur, 2, nullptr, L, L, 0, cur);
            drop(f0);
            quarter(Q2{}, f0, sc, f1, cur, 3, nullptr, L, L, 0, cur);
            drop(f1);
            quarter(Q3{}, f1, sc, f0, cur, -1, nullptr, L, L, 0, cur);
        }
        // no load is on its way to LDS any more, and every wave is done with it
        asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    }

    // Accumulator a of lane l: vector l % 32 of operand a (a row of out), vector
    // 8 (a / 4) + 4 (l / 32) + a % 4 of operand b (a column), of a 32 x 32 block.
    // A wave turns 32 rows at a time around in LDS of its own and stores whole
    // runs of a row.
    constexpr int WC = BN / WN;
    char* const slab = (char*)S + wave * kSlab;
    const int64_t c0 = n0 + wn * WC;
    const int ncol = (int)(p.N - c0 < WC ? p.N - c0 : WC);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const int64_t row0 = m0 + wm * (BM / WM) + 32 * i, row = row0 + lr;
        const int nrow = (int)(mend - row0 < 32 ? mend - row0 : 32);
        float f = 1.0f;
        bool zero = false;
        if constexpr (MODE == GEMM_GROUPED) {
            if (row < mend) {
                if (p.row_scale) f = p.row_scale[row];
                // a row index outside a stands for a row of zeros
                if (p.rows && (uint32_t)p.rows[row] >= (uint64_t)p.A) zero = true;
            }
        }
        auto value = [&](int j, int a) { return zero ? 0.0f : acc[i][j][a] * f; };
        if (p.type == MX_F32) {
            constexpr int W = FN == 1 ? 32 : 64;
            float* const fs = (float*)slab;
#pragma unroll
            for (int j0 = 0; j0 < FN; j0 += 2) {
#pragma unroll
                for (int j = j0; j < j0 + 2 && j < FN; ++j)
#pragma unroll
                    for (int g = 0; g < 4; ++g)
                        *(f32x4*)&fs[lr * (W + 4) + 32 * (j - j0) + 8 * g + 4 * half] =
                            f32x4{value(j, 4 * g), value(j, 4 * g + 1), value(j, 4 * g + 2), value(j, 4 * g + 3)};
                __builtin_amdgcn_wave_barrier();
                store_slab<float, W>(fs, (float*)p.out + out0 + row0 * p.N + c0 + 32 * j0, p.N, nrow, ncol - 32 * j0,
                                     p.N % 4 == 0 && ((uintptr_t)p.out & 15) == 0, lane);
                __builtin_amdgcn_wave_barrier();
            }
        } else {
            uint16_t* const hs = (uint16_t*)slab;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int g = 0; g < 4; ++g)
                    *(u32x2*)&hs[lr * (WC + 8) + 32 * j + 8 * g + 4 * half] =
                        u32x2{pack16(p.type, value(j, 4 * g), value(j, 4 * g + 1)), pack16(p.type, value(j, 4 * g + 2), value(j, 4 * g + 3))};
            __builtin_amdgcn_wave_barrier();
            store_slab<uint16_t, WC>(hs, (uint16_t*)p.out + out0 + row0 * p.N + c0, p.N, nrow, ncol,
                                     p.N % 8 == 0 && ((uintptr_t)p.out & 15) == 0, lane);
            __builtin_amdgcn_wave_barrier();
        }
    }
}

template <int BM, int BN, int WM, int WN, int MODE>
hipError_t launch_tiles(TileArgs p, int64_t mtiles, int64_t batch, hipStream_t st) {
    const int64_t ntn = (p.N + BN - 1) / BN;
    const int64_t grid = mtiles * ntn * batch;
    if (grid > kMxMaxGrid || mtiles > kMxMaxGrid || ntn > kMxMaxGrid) return hipErrorInvalidValue;
    if (grid == 0) return hipSuccess;
    p.ntm = (uint32_t)mtiles;
    p.ntn = (uint32_t)ntn;
    k_mx_gemm<BM, BN, WM, WN, MODE><<<(unsigned)grid, 64 * WM * WN, 0, st>>>(p);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_gemm(const MxGemm& g, hipStream_t st) {
    if (g.M <= 0 || g.N <= 0) return hipSuccess;
    TileArgs p{g.a_q, g.a_sf, g.b_q, g.b_sf, g.A, g.M, g.N, g.Kp / kMxStep, g.out, g.type, g.offsets, g.E, g.M,
               g.rows, g.row_scale, 0, 0};
    if (g.offsets) {
        if (g.M >= 256 * (int64_t)g.E) return launch_tiles<256, 256, 4, 2, GEMM_GROUPED>(p, mx_max_tiles(g.M, g.E, 256), 1, st);
        return launch_tiles<128, 128, 2, 2, GEMM_GROUPED>(p, mx_max_tiles(g.M, g.E, 128), 1, st);
    }
    if (((g.M + 255) / 256) * ((g.N + 255) / 256) >= 256)
        return launch_tiles<256, 256, 4, 2, GEMM_DENSE>(p, (g.M + 255) / 256, 1, st);
    return launch_tiles<128, 128, 2, 2, GEMM_DENSE>(p, (g.M + 127) / 128, 1, st);
}

hipError_t launch_mx_wgrad(const MxWgrad& g, hipStream_t st) {
    if (g.N <= 0 || g.K <= 0 || g.E <= 0) return hipSuccess;
    TileArgs p{g.a_q, g.a_sf, g.b_q, g.b_sf, g.N, g.N, g.K, g.Tp / kMxStep, g.out, g.type, g.offsets, g.E, g.Tp,
               nullptr, nullptr, 0, 0};
    return launch_tiles<128, 128, 2, 2, GEMM_WGRAD>(p, (g.N + 127) / 128, g.E, st);
}

}  // namespace nvfp4
