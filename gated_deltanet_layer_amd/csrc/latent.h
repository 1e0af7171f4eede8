// latent.h -- arguments and shared device helpers of the latent-attention
// kernels (gfx950): latent_fwd.hip, latent_bwd.hip, latent_step.hip.
//
// All of them keep operand tiles in LDS as rows of 16-byte chunks whose index is
// XOR-ed with the row, read matrix-core operands from them either
// along a row (row_frag: contraction over the row's columns) or across rows
// (col_frag: contraction over the rows, through gfx950's transposing LDS read
// for bf16), and hold scores so that an accumulator tile feeds the next product
// as its B operand without leaving the registers (reg_frag).
#pragma once
#include "latent_plan.h"
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
    unsigned page_mul;            // t / page = t page_mul >> page_shift for t < 2^30 (set by the launcher)
    int page_shift;
};

hipError_t latent_fwd_launch(bool bf16, int dn, int dv, const LatentFwdArgs &a, hipStream_t st);
unsigned long long latent_fwd_workspace(bool bf16, int B, int Tq, int Tk, int H, int dv);
hipError_t latent_bwd_launch(bool bf16, int dn, int dv, const LatentBwdArgs &a, hipStream_t st);
unsigned long long latent_bwd_workspace(bool bf16, int B, int Tq, int Tk, int H, int dn, int dv);
hipError_t latent_step_launch(bool bf16, int r, const LatentStepArgs &a, hipStream_t st);
unsigned long long latent_step_workspace(bool bf16, int N, int M, int H, int r);

#ifdef __HIPCC__
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

// Zeros: the source of every tile row behind the last live key, so that what such
// rows hold in memory (it may be NaN) never meets a product.  One row of the widest
// kind (512 + 64 fp32 values).
static __device__ const uint4 latent_zero[144] = {};

// LDS tiles are rows of CPR 16-byte chunks (8, or a multiple of 16); the chunk index
// is XOR-ed with a function of the row.  The LDS serves 16 chunks (64 banks) a clock.
// A 16-byte read goes by groups of 16 lanes, measured as {0-3, 12-15, 20-23, 24-27},
// {4-11, 16-19, 28-31} and the same from 32 on: for row_frag, rows 0-3 and 12-15 at
// one chunk index with rows 4-11 at the next.  col_frag reads eight rows at a pair of
// chunks.  Both fall on 16 distinct slots of 256 bytes if what tells eight rows apart
// moves whole pairs, and the row's bit 3 swaps the chunks of a pair and the halves of
// the eight (with rows XOR-ed by their low bits alone, each row_frag took twice as
// long).  The functions below split an address into a part per lane, computed once,
// and one that folds into the instruction's offset.
template <int CPR> __device__ __forceinline__ constexpr int swz(int row) {
    static_assert(CPR == 8 || CPR % 16 == 0, "");
    return CPR == 8 ? (((row >> 1) & 3) << 1) ^ (((row >> 3) & 1) * 5) : ((row & 7) << 1) ^ (((row >> 3) & 1) * 9);
}

// Keeps what is computed from x where it is used: addresses that the compiler moved out
// of a long loop would stay in registers that the loop needs.
__device__ __forceinline__ int pin(int x) {
    asm volatile("" : "+v"(x));
    return x;
}

// Operand with rows `row` (of this lane) and columns 32 kb + 8 gq .. +7.
template <typename T, int CPR> __device__ __forceinline__ int row_base(int row) {
    const int ch = sizeof(T) == 2 ? lane_gq() : 2 * lane_gq();
    return row * (CPR * 16) + ((ch ^ swz<CPR>(row)) << 4);
}
template <typename T> __device__ __forceinline__ Frag<T> row_frag(const char *M, int base, int kb) {
    if constexpr (sizeof(T) == 2) {
        return {*reinterpret_cast<const bf16x8 *>(M + (base ^ ((kb & 3) << 6)) + (kb >> 2) * 256)};
    } else {
        base ^= (kb & 1) << 7;
        M += (kb >> 1) * 256;
        return {*reinterpret_cast<const f32x4 *>(M + base), *reinterpret_cast<const f32x4 *>(M + (base ^ 16))};
    }
}

// Operand with rows = columns 16 cb + r16 of the tile and contraction slots = tile
// rows row + 0..3 and row + 16 + 0..3 (`row`: 4 gq and a multiple of 16).
template <typename T, int CPR> __device__ __forceinline__ int col_base(int row) {
    const int r16 = lane_r16();
    if constexpr (sizeof(T) == 2) {
        row += r16 >> 2;
        return row * (CPR * 16) + ((((r16 & 3) >> 1) ^ swz<CPR>(row)) << 4) + 8 * (r16 & 1);
    } else {
        return row * (CPR * 16) + (((r16 >> 2) ^ swz<CPR>(row)) << 4) + 4 * (r16 & 3);
    }
}
template <typename T, int CPR> __device__ __forceinline__ Frag<T> col_frag(const char *M, int base, int cb) {
    if constexpr (sizeof(T) == 2) {
        const char *m = M + (base ^ ((cb & 7) << 5)) + (cb >> 3) * 256;
        return {cat8(lds_read_tr(lds_u32(m)), lds_read_tr(lds_u32(m + 16 * CPR * 16)))};
    } else {
        static_assert(CPR % 16 == 0, "");
        const int at = base ^ ((cb & 3) << 6);
        const char *m = M + (cb >> 2) * 256;
        Frag<T> f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {   // row + e: bits 1 and 2 of the chunk index
            f.lo[e] = *reinterpret_cast<const float *>(m + (at ^ (e << 5)) + e * CPR * 16);
            f.hi[e] = *reinterpret_cast<const float *>(m + (at ^ (e << 5)) + (16 + e) * CPR * 16);
        }
        return f;
    }
}

// Copies into LDS for the middle of other work: as g2lds16, g2lds16s and g2lds4, but
// without the memory clobber, so that LDS reads of other buffers may move across them
// (they keep their order among themselves and to the waits and barriers, which are
// volatile too), and with addresses that the caller has in scalar registers.
__device__ __forceinline__ unsigned lds_at(const char *lds) {   // uniform
    return (unsigned)(uintptr_t)(__attribute__((address_space(3))) const char *)lds;
}
__device__ __forceinline__ void copy16(const void *src, const char *lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(src), "s"(lds_at(lds)) : "m0");
}
// base: uniform, and from scalar instructions or settled (below).
__device__ __forceinline__ void copy16s(const void *base, unsigned off, const char *lds) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds_at(lds)) : "m0");
}
// Address that lane `lane` holds, in scalar registers, and the wait for a group of them:
// a memory instruction reads a scalar register that a vector instruction wrote five wait
// states later at the soonest, and the compiler does not see the loads in the copies.  The
// operands tie it between the lane reads and the copies.
__device__ __forceinline__ unsigned long long lane_address(const char *p, int lane) {
    const unsigned lo = (unsigned)__builtin_amdgcn_readlane((int)(uintptr_t)p, lane);
    const unsigned hi = (unsigned)__builtin_amdgcn_readlane((int)((uintptr_t)p >> 32), lane);
    return (unsigned long long)hi << 32 | lo;
}
__device__ __forceinline__ void settle(unsigned long long (&b)[8]) {
    asm volatile("s_nop 4" : "+s"(b[0]), "+s"(b[1]), "+s"(b[2]), "+s"(b[3]), "+s"(b[4]), "+s"(b[5]), "+s"(b[6]), "+s"(b[7]));
}
__device__ __forceinline__ void copy4(const void *src, const char *lds) {
    asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(src), "s"(lds_at(lds)) : "m0");
}

// Enqueue the copy of rows r0 .. r0 + ROWS - 1 (CPR chunks each, `stride` bytes
// apart, x: row 0) into an LDS tile by NTHR threads; rows from n on read as zeros.
// One instruction of the workgroup covers NTHR / CPR rows, a multiple of 8, so the
// lane's offset within them is the same for all, but for row bit 3 where it is 8.
template <int CPR, int ROWS, int NTHR = 256>
__device__ __forceinline__ void load_rows(char *tile, const char *x, long stride, int r0, int n)
{
    constexpr int RP = NTHR / CPR;
    static_assert(RP % 8 == 0 && ROWS % RP == 0, "");
    const int tid = threadIdx.x, row = tid / CPR, ch = ((tid % CPR) ^ swz<CPR>(row)) * 16;
    const char *dst = tile + __builtin_amdgcn_readfirstlane(tid >> 6) * 1024, *p = x + r0 * stride;
    if (r0 + ROWS <= n) {
        const unsigned off = (unsigned)(row * (int)stride + ch);
#pragma unroll
        for (int i = 0; i < ROWS / RP; ++i)
            copy16s(p + i * RP * stride, RP == 8 && (i & 1) ? (unsigned)(row * (int)stride + (ch ^ 144)) : off, dst + i * NTHR * 16);
    } else {
#pragma unroll
        for (int i = 0; i < ROWS / RP; ++i) {
            const char *src = r0 + i * RP + row < n ? p + (i * RP + row) * stride + (RP == 8 && (i & 1) ? ch ^ 144 : ch)
                                                    : (const char *)latent_zero;
            copy16(src, dst + i * NTHR * 16);
        }
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

// Order for the scheduler: AHEAD LDS reads, then after every group of M matrix
// products R more reads, as long as reads are left.  Left to itself the compiler puts
// each read right before its product and waits for it there.
template <int AHEAD, int READS, int PRODUCTS, int R, int M> __device__ __forceinline__ void pipeline() {
    __builtin_amdgcn_sched_group_barrier(0x100, AHEAD, 0);
#pragma unroll
    for (int i = AHEAD; i < READS; i += R) {
        __builtin_amdgcn_sched_group_barrier(0x008, M, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, R, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, PRODUCTS, 0);
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
