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

#include "nvfp4_mx.hpp"

namespace nvfp4 {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kFp4 = 4;   // the MFMA's format selector for E2M1

// the MFMA's operand registers: an FP4 operand uses the first four
__device__ __forceinline__ i32x8 frag(u32x4 v) { return i32x8{(int)v.x, (int)v.y, (int)v.z, (int)v.w, 0, 0, 0, 0}; }

__device__ __forceinline__ void store_out(void* out, int type, int64_t i, float v) {
    if (type == MX_F32) ((float*)out)[i] = v;
    else if (type == MX_BF16) ((uint16_t*)out)[i] = (uint16_t)bf16x2_rne(v, 0.0f);
    else ((_Float16*)out)[i] = (_Float16)v;
}

// ------------------------------------------------------------ many rows
//
// A workgroup of WM x WN waves computes a BM x BN tile in steps of 128
// elements: 64 code bytes and one scale word per operand row, brought to LDS
// by loads that go there directly, kStages steps in rotation.  A wave keeps
// (BM / WM) x (BN / WN) of the tile in 32 x 32 accumulators; v_mfma_scale
// 32x32x64 takes row l % 32 of either operand in lane l, lanes 0-31 one block
// and lanes 32-63 another: blocks 0, 1 of the step in the lower half and 2, 3
// in the upper, so that a lane's two scales are adjacent bytes.
//
// LDS: row r's four 16-byte chunks at 64 r, chunk c in place c ^ (r / 2 % 4):
// 8 lanes reading one chunk of 8 rows touch all the banks once.

enum GemmMode { GEMM_DENSE, GEMM_GROUPED, GEMM_WGRAD };

constexpr int kStages = 3;

template <int BM, int BN>
struct GemmStage {
    uint8_t q[(BM + BN) * 64];
    uint32_t sf[BM + BN];
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

template <int BM, int BN, int WM, int WN, int MODE>
__global__ __launch_bounds__(64 * WM * WN) void k_mx_gemm(TileArgs p) {
    constexpr int NT = 64 * WM * WN, FM = BM / WM / 32, FN = BN / WN / 32;
    constexpr int QL = (BM + BN) * 4 / NT;        // 16-byte chunks a thread brings per step
    static_assert((BM + BN) * 4 % NT == 0 && (BM + BN) <= NT && BM % 64 == 0, "");
    __shared__ __attribute__((aligned(16))) GemmStage<BM, BN> S[kStages];
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / WN, wn = wave % WN;

    int64_t m0, n0, mend = p.M, step0 = 0, steps = p.Kt, out0 = 0;
    const uint8_t *b_q = p.b_q, *b_sf = p.b_sf;
    {
        uint32_t id = blockIdx.x;
        if constexpr (MODE == GEMM_WGRAD) {
            const uint32_t per = p.ntm * p.ntn;
            const int e = (int)(id / per);
            id -= (uint32_t)e * per;
            // the group's steps in the padded rows follow those of the groups before it
            int64_t before = 0;
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
            step0 = __builtin_amdgcn_readfirstlane((int)before);
            steps = (b - a + 127) >> 7;
            // offsets that are not in order could ask for more steps than there are
            if (step0 + steps > p.Kt) steps = p.Kt > step0 ? p.Kt - step0 : 0;
            out0 = (int64_t)e * p.M * p.N;
        }
        m0 = (int64_t)(id / p.ntn) * BM;
        n0 = (int64_t)(id % p.ntn) * BN;
        if constexpr (MODE == GEMM_GROUPED) {
            const MxGroupTile g = mx_find_group(p.offsets, p.E, p.R, BM, id / p.ntn);
            if (g.e < 0) return;
            m0 = g.begin;
            mend = g.end;
            b_q += (int64_t)g.e * p.N * p.Kt * 64;
            b_sf += (int64_t)g.e * ((p.N + 127) / 128) * p.Kt * 512;
        }
    }

    // what this thread brings each step: sources for step `step0`
    const uint8_t* qsrc[QL];
#pragma unroll
    for (int i = 0; i < QL; ++i) {
        const int slot = tid + NT * i, r = slot >> 2, c = (slot & 3) ^ ((r >> 1) & 3);
        const uint8_t* base;
        int64_t row;
        if (r < BM) {
            row = m0 + r < mend ? m0 + r : mend - 1;
            if constexpr (MODE == GEMM_GROUPED) {
                if (p.rows) row = p.rows[row];
                row = row < 0 ? 0 : (row < p.A ? row : p.A - 1);
            }
            base = p.a_q;
        } else {
            row = n0 + r - BM < p.N ? n0 + r - BM : p.N - 1;
            base = b_q;
        }
        qsrc[i] = base + (row * p.Kt + step0) * 64 + 16 * c;
    }
    const uint8_t* ssrc;
    {
        const int r = tid < BM + BN ? tid : BM + BN - 1;
        int64_t row;
        if (r < BM) {
            row = m0 + r < mend ? m0 + r : mend - 1;
            if constexpr (MODE == GEMM_GROUPED) {
                if (p.rows) row = p.rows[row];
                row = row < 0 ? 0 : (row < p.A ? row : p.A - 1);
            }
        } else {
            row = n0 + r - BM < p.N ? n0 + r - BM : p.N - 1;
        }
        ssrc = (r < BM ? p.a_sf : b_sf) + mx_sf_offset(row, step0, p.Kt);
    }
    const bool brings_sf = (BM + BN) % 64 == 0 && 64 * wave < BM + BN;
    auto bring = [&](int64_t s) {
        // past the last step the last one comes again, into a stage nobody reads
        const int64_t k = s < steps ? s : steps - 1;
        GemmStage<BM, BN>& st = S[s % kStages];
#pragma unroll
        for (int i = 0; i < QL; ++i) load16_to_lds(qsrc[i] + k * 64, &st.q[16 * (64 * wave + NT * i)]);
        if (brings_sf) load4_to_lds(ssrc + k * 512, &st.sf[64 * wave]);
    };

    f32x16 acc[FM][FN];
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int a = 0; a < 16; ++a) acc[i][j][a] = 0.0f;

    const int half = lane >> 5, lr = lane & 31;
    if (steps > 0) {
        for (int s = 0; s < kStages - 1; ++s) bring(s);
        for (int64_t s = 0; s < steps; ++s) {
            // step s has landed when at most the later steps' loads are out, and
            // this wave has read all of step s - 1, whose stage is written next
            if (brings_sf) asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kStages - 2) * (QL + 1)) : "memory");
            else asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kStages - 2) * QL) : "memory");
            asm volatile("s_barrier" ::: "memory");
            bring(s + kStages - 1);
            const GemmStage<BM, BN>& st = S[s % kStages];
            int sa[FM], sb[FN];
#pragma unroll
            for (int i = 0; i < FM; ++i)
                sa[i] = ((const uint16_t*)&st.sf[wm * (BM / WM) + 32 * i + lr])[half];
#pragma unroll
            for (int j = 0; j < FN; ++j)
                sb[j] = ((const uint16_t*)&st.sf[BM + wn * (BN / WN) + 32 * j + lr])[half];
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                u32x4 a[FM], b[FN];
                const int c = (2 * half + kk) ^ ((lr >> 1) & 3);
#pragma unroll
                for (int i = 0; i < FM; ++i)
                    a[i] = *(const u32x4*)&st.q[(wm * (BM / WM) + 32 * i + lr) * 64 + 16 * c];
#pragma unroll
                for (int j = 0; j < FN; ++j)
                    b[j] = *(const u32x4*)&st.q[(BM + wn * (BN / WN) + 32 * j + lr) * 64 + 16 * c];
#pragma unroll
                for (int i = 0; i < FM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j) {
                        if (kk == 0)
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                frag(a[i]), frag(b[j]), acc[i][j], kFp4, kFp4, 0, sa[i], 0, sb[j]);
                        else
                            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                frag(a[i]), frag(b[j]), acc[i][j], kFp4, kFp4, 1, sa[i], 1, sb[j]);
                    }
            }
        }
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }

    // accumulator a of lane l: row 8 (a / 4) + 4 (l / 32) + a % 4, column l % 32
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int a = 0; a < 16; ++a) {
            const int64_t row = m0 + wm * (BM / WM) + 32 * i + 8 * (a >> 2) + 4 * half + (a & 3);
            if (row >= mend) continue;
            float f = 1.0f;
            bool zero = steps <= 0;
            if constexpr (MODE == GEMM_GROUPED) {
                if (p.row_scale) f = p.row_scale[row];
                // a row index outside a stands for a row of zeros
                if (p.rows && (uint32_t)p.rows[row] >= (uint64_t)p.A) zero = true;
            }
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                const int64_t col = n0 + wn * (BN / WN) + 32 * j + lr;
                if (col < p.N) store_out(p.out, p.type, out0 + row * p.N + col, zero ? 0.0f : acc[i][j][a] * f);
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
    if (g.offsets) return launch_tiles<128, 128, 2, 2, GEMM_GROUPED>(p, mx_max_tiles(g.M, g.E, 128), 1, st);
    return launch_tiles<128, 128, 2, 2, GEMM_DENSE>(p, (g.M + 127) / 128, 1, st);
}

hipError_t launch_mx_wgrad(const MxWgrad& g, hipStream_t st) {
    if (g.N <= 0 || g.K <= 0 || g.E <= 0) return hipSuccess;
    TileArgs p{g.a_q, g.a_sf, g.b_q, g.b_sf, g.N, g.N, g.K, g.Tp / kMxStep, g.out, g.type, g.offsets, g.E, g.Tp,
               nullptr, nullptr, 0, 0};
    return launch_tiles<128, 128, 2, 2, GEMM_WGRAD>(p, (g.N + 127) / 128, g.E, st);
}

}  // namespace nvfp4
