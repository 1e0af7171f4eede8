// attn_prologue.hip -- norms of query and key heads with the rotation by position, and
// their gradients (gfx950).
//
//   x' = w x r,  r = 1 / sqrt(mean_c x_c^2 + eps)                 (per token and head)
//   y_i = x'_i cos a_i - x'_{i+R/2} sin a_i,  y_{i+R/2} = x'_{i+R/2} cos a_i + x'_i sin a_i
//   a_i = pos inv_freq_i, i < R/2; channels from R on stay as x'
//
// With z = the gradient of y turned back by the same angles:
//   dw_c = sum over tokens and heads of z_c x_c r,  dx = r (w z - x r mean(w z x r))
//
// Bound by HBM: every value is read once and written once.  A workgroup takes a few
// tokens, works out their cosines and sines once for all heads (the angle in turns in
// 64 bits, its fraction to fp32: at position 10^6 an fp32 product would be off by 0.06
// radians), and then goes through the heads, D / 8 lanes a head with eight channels each.
// A lane reads the partners of its channels itself: they are in the lines that its
// neighbours read.  16384 tokens of 32 and 8 heads of 128 in bf16 (336 MB) take 69 us, 4.9 TB/s
// (66 to 71 in single calls); their gradients (504 MB) 98 us, of which the last kernel, the sums of dw, 5.
#include "attn.h"

namespace gdn {

template <typename T> struct Eight {
    float v[8];
    __device__ __forceinline__ void load(const T *p) {
        if constexpr (sizeof(T) == 2) {
            const bf16x8 x = *reinterpret_cast<const bf16x8 *>(p);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (float)x[e];
        } else {
            const f32x4 a = *reinterpret_cast<const f32x4 *>(p), b = *reinterpret_cast<const f32x4 *>(p + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
        }
    }
    __device__ __forceinline__ void store(T *p) const {
        store4(p, f32x4{v[0], v[1], v[2], v[3]});
        store4(p + 4, f32x4{v[4], v[5], v[6], v[7]});
    }
};
template <> __device__ __forceinline__ void Eight<__bf16>::store(__bf16 *p) const {
    *reinterpret_cast<bf16x8 *>(p) = cat8(cvt4(f32x4{v[0], v[1], v[2], v[3]}), cvt4(f32x4{v[4], v[5], v[6], v[7]}));
}

// Sum over the LPH lanes of a head (8 or 16), in all of them.
template <int LPH> __device__ __forceinline__ float head_sum(float x) {
#pragma unroll
    for (int d = 1; d < LPH; d <<= 1) x += __shfl_xor(x, d, LPH);
    return x;
}

// Cosines and sines of TPW tokens in LDS, [TPW][2][R / 2].
template <int TPW> __device__ __forceinline__ void turn(float *cs, const AttnPrologueArgs &a, int t0)
{
    const int h = a.R / 2;
    for (int i = threadIdx.x; i < TPW * h; i += 256) {
        const int t = i / h, f = i - t * h;
        if (t0 + t >= a.T) break;
        const double turns = (double)a.pos[t0 + t] * ((double)a.inv_freq[f] * 0.15915494309189535);
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[t * 2 * h + f] = c;
        cs[t * 2 * h + h + f] = s;
    }
    __syncthreads();
}

// Channels of a lane: its own eight, their partners', and the cosines and sines between.
template <int D> struct Lane {
    int at, other;      // first channel, first partner (itself where not rotated)
    float cos[8], sin[8];
    __device__ __forceinline__ Lane(const float *cs, int t, int R) {
        const int h = R / 2;
        at = threadIdx.x % (D / 8) * 8;
        const bool turned = at < R, low = at < h;
        other = !turned ? at : low ? at + h : at - h;
        const float *p = cs + t * R + (low ? at : at - h);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            cos[e] = turned ? p[e] : 1.f;
            sin[e] = !turned ? 0.f : low ? -p[h + e] : p[h + e];
        }
    }
};

template <typename T, int D, int TPW> __global__ __launch_bounds__(256) void attn_prologue_kernel(AttnPrologueArgs a)
{
    constexpr int LPH = D / 8, GROUPS = 256 / LPH / TPW;   // heads at a time of each token
    __shared__ float cs[TPW * D];
    const int t0 = blockIdx.x * TPW;
    turn<TPW>(cs, a, t0);
    const int group = threadIdx.x / LPH, tl = group / GROUPS, first = group % GROUPS;
    const long t = t0 + tl;
    if (t >= a.T) return;
    const Lane<D> ln(cs, tl, a.R);
    auto heads = [&](const T *x, const float *w, T *y, int H) {
        if (first >= H) return;
        Eight<float> wo, wp;
        wo.load(w + ln.at);
        wp.load(w + ln.other);
        for (int h = first; h < H; h += GROUPS) {
            Eight<T> o, p;
            o.load(x + h * D + ln.at);
            p.load(x + h * D + ln.other);
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s += o.v[e] * o.v[e];
            const float r = 1.f / sqrtf(head_sum<LPH>(s) * (1.f / D) + a.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) o.v[e] = o.v[e] * r * wo.v[e] * ln.cos[e] + p.v[e] * r * wp.v[e] * ln.sin[e];
            o.store(y + h * D + ln.at);
        }
    };
    heads((const T *)a.q_raw + t * a.q_stride, a.w_q, (T *)a.q + t * a.Hq * D, a.Hq);
    heads((const T *)a.k_raw + t * a.k_stride, a.w_k, (T *)a.k + t * a.Hk * D, a.Hk);
}

// Tokens at a time of a workgroup, and the workgroups: up to four a compute unit, which share
// the tokens.  One token where there is one for each, if it has heads for all lanes (32 over 8
// heads of 128, bf16: 64 tokens 7.3 us, four at a time 10.7; 1024 13.1, 14.6) or the call is
// short (16 over 2 of 64: 64 tokens 6.7 us, 7.3; 512 9.2, 7.7); above, four (32 over 8 heads,
// 4096 tokens 26.1 us, one at a time 27.9; with 512 workgroups 28.6, with 2048 26.0 and, of
// 16384 tokens, 113.8 and 100.4 for 98.9).
constexpr int PRO_BWD_WGS = 1024;
static int pro_bwd_tokens(int T, int Hq, int D) { return T <= (Hq * D >= 4096 ? PRO_BWD_WGS : 128) ? 1 : 4; }
static int pro_bwd_wgs(int T, int tokens) {
    const int n = (T + tokens - 1) / tokens;
    return n < PRO_BWD_WGS ? n : PRO_BWD_WGS;
}

// Sums of dw: each lane adds up its channels over the tokens of its workgroup, the
// workgroup its groups' sums, and attn_prologue_dw_kernel the workgroups', all in order.
template <typename T, int D, int TPW> __global__ __launch_bounds__(256) void attn_prologue_bwd_kernel(AttnPrologueArgs a)
{
    constexpr int LPH = D / 8, NG = 256 / LPH, GROUPS = NG / TPW;
    __shared__ float cs[TPW * D];
    __shared__ float sums[NG][D];
    const int group = threadIdx.x / LPH, tl = group / GROUPS, first = group % GROUPS;
    float dw[2][8] = {};
    for (int t0 = blockIdx.x * TPW; t0 < a.T; t0 += gridDim.x * TPW) {
        __syncthreads();   // the tokens before are done with
        turn<TPW>(cs, a, t0);
        const long t = t0 + tl;
        if (t >= a.T) continue;
        const Lane<D> ln(cs, tl, a.R);
        auto heads = [&](const T *x, const T *dy, const float *w, T *dx, int H, float (&dw)[8]) {
            if (first >= H) return;
            Eight<float> wo;
            wo.load(w + ln.at);
            for (int h = first; h < H; h += GROUPS) {
                Eight<T> o, z, p;
                o.load(x + h * D + ln.at);
                z.load(dy + h * D + ln.at);
                p.load(dy + h * D + ln.other);
                float s = 0.f, m = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    s += o.v[e] * o.v[e];
                    z.v[e] = z.v[e] * ln.cos[e] - p.v[e] * ln.sin[e];
                    m += wo.v[e] * z.v[e] * o.v[e];
                }
                const float r = 1.f / sqrtf(head_sum<LPH>(s) * (1.f / D) + a.eps);
                const float c = head_sum<LPH>(m) * (1.f / D) * r * r;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    dw[e] += z.v[e] * o.v[e] * r;
                    o.v[e] = r * (wo.v[e] * z.v[e] - o.v[e] * c);
                }
                o.store(dx + h * D + ln.at);
            }
        };
        heads((const T *)a.q_raw + t * a.q_stride, (const T *)a.q + t * a.Hq * D, a.w_q, (T *)a.dq_raw + t * a.dq_stride, a.Hq, dw[0]);
        heads((const T *)a.k_raw + t * a.k_stride, (const T *)a.k + t * a.Hk * D, a.w_k, (T *)a.dk_raw + t * a.dk_stride, a.Hk, dw[1]);
    }
    const int at = threadIdx.x % LPH * 8;
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[group][at + e] = dw[n][e];
        __syncthreads();
        if (threadIdx.x < D) {
            float s = 0.f;
#pragma unroll
            for (int g = 0; g < NG; ++g) s += sums[g][threadIdx.x];
            a.ws[((long)blockIdx.x * 2 + n) * D + threadIdx.x] = s;
        }
    }
}

// dw_q and dw_k from the workgroups' sums: a workgroup for 16 channels, 64 runs of the sums.
template <int D> __global__ __launch_bounds__(1024) void attn_prologue_dw_kernel(AttnPrologueArgs a, int wgs)
{
    __shared__ float sums[64][16];
    const int c = threadIdx.x & 15, run = threadIdx.x >> 4, col = blockIdx.x * 16 + c;   // of 2 D columns
    const int per = (wgs + 63) / 64, end = min(wgs, (run + 1) * per);
    float s = 0.f;
#pragma unroll 16
    for (int i = run * per; i < end; ++i) s += a.ws[(long)i * 2 * D + col];
    sums[run][c] = s;
    __syncthreads();
    if (run > 0) return;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 64; ++i) s += sums[i][c];
    (col < D ? a.dw_q : a.dw_k)[col % D] = s;
}

// Four tokens a workgroup once that leaves workgroups for four a compute unit (32 over 8 heads
// of 128, bf16: 64 tokens 4.3 us one a workgroup, 7.7 four; 2048 11.1, 11.8; 4096 18.0, 16.2;
// 16384 76, 69, which is 4.9 TB/s).
template <typename T, int D> static hipError_t prologue(const AttnPrologueArgs &a, hipStream_t st)
{
    if (a.T >= 4096) hipLaunchKernelGGL((attn_prologue_kernel<T, D, 4>), dim3((a.T + 3) / 4), dim3(256), 0, st, a);
    else hipLaunchKernelGGL((attn_prologue_kernel<T, D, 1>), dim3(a.T), dim3(256), 0, st, a);
    return hipGetLastError();
}

template <typename T, int D> static hipError_t prologue_bwd(const AttnPrologueArgs &a, hipStream_t st)
{
    const int tokens = pro_bwd_tokens(a.T, a.Hq, D), wgs = pro_bwd_wgs(a.T, tokens);
    if (wgs > 0 && tokens == 1) hipLaunchKernelGGL((attn_prologue_bwd_kernel<T, D, 1>), dim3(wgs), dim3(256), 0, st, a);
    else if (wgs > 0) hipLaunchKernelGGL((attn_prologue_bwd_kernel<T, D, 4>), dim3(wgs), dim3(256), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((attn_prologue_dw_kernel<D>), dim3(2 * D / 16), dim3(1024), 0, st, a, wgs);
    return hipGetLastError();
}

hipError_t attn_prologue_launch(bool bf16, int D, const AttnPrologueArgs &a, hipStream_t st)
{
    if (bf16) return D == 128 ? prologue<__bf16, 128>(a, st) : prologue<__bf16, 64>(a, st);
    return D == 128 ? prologue<float, 128>(a, st) : prologue<float, 64>(a, st);
}

hipError_t attn_prologue_bwd_launch(bool bf16, int D, const AttnPrologueArgs &a, hipStream_t st)
{
    if (bf16) return D == 128 ? prologue_bwd<__bf16, 128>(a, st) : prologue_bwd<__bf16, 64>(a, st);
    return D == 128 ? prologue_bwd<float, 128>(a, st) : prologue_bwd<float, 64>(a, st);
}

unsigned long long attn_prologue_bwd_workspace(int T, int Hq, int D)
{
    return (unsigned long long)pro_bwd_wgs(T, pro_bwd_tokens(T, Hq, D)) * 2 * D * 4;
}

} // namespace gdn
