// latent.h -- arguments and shared device helpers of the latent-attention
// kernels (gfx950): latent_fwd.hip, latent_bwd.hip, latent_step.hip.
//
// All of them keep operand tiles in LDS as rows of 16-byte chunks whose index is
// XOR-ed with the row (latent_off), read matrix-core operands from them either
// along a row (row_frag: contraction over the row's columns) or across rows
// (col_frag: contraction over the rows, through gfx950's transposing LDS read
// for bf16), and hold scores so that an accumulator tile feeds the next product
// as its B operand without leaving the registers (reg_frag).
#pragma once
#include "ws_common.h"
#include <stddef.h>

namespace gdn {

constexpr int LATENT_ROPE = 64;   // width of the rotary key that all heads share
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

struct LatentFwdArgs {
    const void *q, *kv, *k_rope;
    const int *lens;
    void *o;
    float *lse;
    void *ws;
    float scale;
    int B, Tq, Tk, H;
};

struct LatentBwdArgs {
    const void *q, *kv, *k_rope;
    const int *lens;
    const void *o;
    const float *lse;
    const void *d_o;
    void *dq, *dkv, *dk_rope;
    void *ws;
    float scale;
    int B, Tq, Tk, H;
};

struct LatentStepArgs {
    const void *q, *draft;
    const long long *tree;
    const void *cache;
    const int *table, *lens;
    void *o;
    float *lse;
    void *ws;
    float scale;
    int N, M, H, drafts;          // drafts: M, or 0 without drafted rows
    int pages, page, width;       // pages in the cache, tokens a page, table columns
};

hipError_t latent_fwd_launch(bool bf16, int dn, int dv, const LatentFwdArgs &a, hipStream_t st);
unsigned long long latent_fwd_workspace(bool bf16, int B, int Tq, int Tk, int H, int dv);
hipError_t latent_bwd_launch(bool bf16, int dn, int dv, const LatentBwdArgs &a, hipStream_t st);
unsigned long long latent_bwd_workspace(int B, int Tq, int Tk, int H);
hipError_t latent_step_launch(bool bf16, int r, const LatentStepArgs &a, hipStream_t st);
unsigned long long latent_step_workspace(bool bf16, int N, int M, int H, int r);

#ifdef __HIPCC__
// Sixteen zero bytes: the source of every tile row behind the last live key, so
// that what such rows hold in memory (it may be NaN) never meets a product.
static __device__ const uint4 latent_zero = {0u, 0u, 0u, 0u};

// Byte offset of the 16-byte chunk `ch` of row `row`, rows of CPR chunks (a
// multiple of 8): the low three bits of the chunk index are XOR-ed with the row,
// so that eight rows read at one chunk index fall on distinct banks.
template <int CPR> __device__ __forceinline__ int latent_off(int row, int ch) {
    static_assert(CPR % 8 == 0, "rows are a multiple of 128 bytes");
    return row * (CPR * 16) + ((ch ^ (row & 7)) << 4);
}

// Operand with rows row0 + r16 and columns 32 kb + 8 gq .. +7.
template <typename T, int CPR> __device__ __forceinline__ Frag<T> row_frag(const char *M, int row0, int kb);
template <int CPR> __device__ __forceinline__ Frag<__bf16> row_frag_bf(const char *M, int row0, int kb) {
    return {*reinterpret_cast<const bf16x8 *>(M + latent_off<CPR>(row0 + lane_r16(), 4 * kb + lane_gq()))};
}
template <int CPR> __device__ __forceinline__ Frag<float> row_frag_f(const char *M, int row0, int kb) {
    const int row = row0 + lane_r16(), ch = 8 * kb + 2 * lane_gq();
    return {*reinterpret_cast<const f32x4 *>(M + latent_off<CPR>(row, ch)),
            *reinterpret_cast<const f32x4 *>(M + latent_off<CPR>(row, ch + 1))};
}
template <typename T, int CPR> __device__ __forceinline__ Frag<T> row_frag(const char *M, int row0, int kb) {
    if constexpr (sizeof(T) == 2) return row_frag_bf<CPR>(M, row0, kb);
    else return row_frag_f<CPR>(M, row0, kb);
}

// Operand with rows = columns 16 cb + r16 of the tile and contraction slots =
// tile rows rowA + 0..3, rowB + 0..3 (rowA and rowB of this lane's group,
// multiples of 4).
template <typename T, int CPR>
__device__ __forceinline__ Frag<T> col_frag(const char *M, int rowA, int rowB, int cb) {
    const int r16 = lane_r16();
    if constexpr (sizeof(T) == 2) {
        const int ch = 2 * cb + ((r16 & 3) >> 1), sub = 8 * (r16 & 1), dr = r16 >> 2;
        return {cat8(lds_read_tr(lds_u32(M + latent_off<CPR>(rowA + dr, ch) + sub)),
                     lds_read_tr(lds_u32(M + latent_off<CPR>(rowB + dr, ch) + sub)))};
    } else {
        const int ch = 4 * cb + (r16 >> 2), sub = 4 * (r16 & 3);
        Frag<T> f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            f.lo[e] = *reinterpret_cast<const float *>(M + latent_off<CPR>(rowA + e, ch) + sub);
            f.hi[e] = *reinterpret_cast<const float *>(M + latent_off<CPR>(rowB + e, ch) + sub);
        }
        return f;
    }
}

// Operand straight from global memory: 8 values of this lane's row.
template <typename T> __device__ __forceinline__ Frag<T> load_frag(const T *p) {
    if constexpr (sizeof(T) == 2) return {*reinterpret_cast<const bf16x8 *>(p)};
    else return {*reinterpret_cast<const f32x4 *>(p), *reinterpret_cast<const f32x4 *>(p + 4)};
}
template <typename T> __device__ __forceinline__ Frag<T> zero_frag() {
    Frag<T> f;
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f.v[e] = (__bf16)0.f;
    } else {
        f.lo = f32x4{0.f, 0.f, 0.f, 0.f};
        f.hi = f.lo;
    }
    return f;
}

template <typename T> __device__ __forceinline__ void store4(T *p, f32x4 v) {
    if constexpr (sizeof(T) == 2) *reinterpret_cast<bf16x4 *>(p) = cvt4(v);
    else *reinterpret_cast<f32x4 *>(p) = v;
}

// Maximum and sum over the four 16-lane rows of a wave, per lane of a row.
__device__ __forceinline__ float rows_max(float x) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_int(x), __float_as_int(x), false, false);
    x = fmaxf(__int_as_float((int)a[0]), __int_as_float((int)a[1]));
    a = __builtin_amdgcn_permlane32_swap(__float_as_int(x), __float_as_int(x), false, false);
    return fmaxf(__int_as_float((int)a[0]), __int_as_float((int)a[1]));
}
__device__ __forceinline__ float rows_sum(float x) {
    auto a = __builtin_amdgcn_permlane16_swap(__float_as_int(x), __float_as_int(x), false, false);
    x = __int_as_float((int)a[0]) + __int_as_float((int)a[1]);
    a = __builtin_amdgcn_permlane32_swap(__float_as_int(x), __float_as_int(x), false, false);
    return __int_as_float((int)a[0]) + __int_as_float((int)a[1]);
}

// 2^x by the hardware's instruction (1 ulp; results below the normal range go to 0).
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// A running maximum is raised only when a score passes it by more than this many
// powers of two: weights stay below 2^8 and their fp32 sums lose nothing, while
// most tiles need no rescaling of the accumulators.
constexpr float RAISE = 8.f;

// Live length of a padded sequence.
__device__ __forceinline__ int live_len(const int *lens, int b, int full) {
    if (!lens) return full;
    const int n = lens[b];
    return n < 0 ? 0 : n > full ? full : n;
}
#endif

} // namespace gdn
