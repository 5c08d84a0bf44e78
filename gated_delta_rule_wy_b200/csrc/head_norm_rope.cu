// head_norm_rope.cu -- the norm of queries and keys per head and the rotation by position,
// in one pass, and its gradients:
//
//   xh = x / r,  r = sqrt(mean_j x_j^2 + eps) (rms), sqrt(sum_j x_j^2 + eps) (l2) or 1
//   v = xh (.) weight;  of the first R channels each pair (v_a, v_b) turns by the position's angle:
//   y_a = v_a cos - v_b sin,  y_b = v_b cos + v_a sin;  pairs (j, j + R / 2) or (2 j, 2 j + 1)
//   backward: dv = dy turned back;  dweight = sum dv (.) xh;  g = dv (.) weight;
//             dx = (g - xh (xh . g) / (d or 1)) / r
//
// Cosines and sines come from a table [positions][R], made by the caller in as many bits as
// far positions need. An HBM stream: one read and one write per element (two reads and one
// write backward). d / 8 lanes own a row of d channels, eight channels each; they walk over
// the heads of one token, so that its angles are read once and stay in registers.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr2_launch.h"
#include "seq_ops.h"

namespace gdr2 {
namespace {

using namespace seq;

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 1024;  // of the backward: one partial weight gradient each
constexpr int kHeads = 4;         // heads in flight per group

struct Side {
    int H, chunks;  // heads, tasks per token
    const void *x, *dy;
    long long ld;
    const float *weight;
    void *out;
};

struct NormParams {
    long long tokens, tasks;
    int T, R, P, first, per;  // per: heads per task
    int norm;
    bool interleaved;
    float eps;
    const float *cos_sin;
    const int *positions;
    Side side[2];
    float *part;  // backward: [blocks][2][d]
    unsigned *status;
};

// The angles of one position for channels 8 l .. 8 l + 7 of a row: cosine and the signed sine
// with which the partner channel enters (y_a: -sin, y_b: +sin).
template <int D>
__device__ __forceinline__ void load_angles(const NormParams &p, long long token, int l, float (&cs)[8], float (&sn)[8])
{
#pragma unroll
    for (int i = 0; i < 8; ++i) { cs[i] = 1.f; sn[i] = 0.f; }
    if (8 * l >= p.R) return;
    const int pos = p.positions ? __ldg(p.positions + token) : p.first + (int)(token % p.T);
    if (pos < 0 || pos >= p.P) {  // reported; the row keeps its norm and is not turned
        atomicOr(p.status, kStatusBadPosition);
        return;
    }
    const float *row = p.cos_sin + (size_t)pos * p.R;
    const int half = p.R / 2;
    if (p.interleaved) {
        const float4 c = __ldg(reinterpret_cast<const float4 *>(row + 4 * l));
        const float4 s = __ldg(reinterpret_cast<const float4 *>(row + half + 4 * l));
        const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) { cs[i] = cc[i / 2]; sn[i] = (i & 1) ? ss[i / 2] : -ss[i / 2]; }
    } else {
        const bool upper = 8 * l >= half;
        const float *c = row + 8 * l - (upper ? half : 0), *s = c + half;
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            const float4 a = __ldg(reinterpret_cast<const float4 *>(c + i));
            const float4 b = __ldg(reinterpret_cast<const float4 *>(s + i));
            const float cc[4] = {a.x, a.y, a.z, a.w}, ss[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) { cs[i + k] = cc[k]; sn[i + k] = upper ? ss[k] : -ss[k]; }
        }
    }
}

// y_i = v_i cos_i + v_partner sin_i over a row (sign = -1 turns back)
__device__ __forceinline__ void turn(float (&v)[8], const float (&cs)[8], const float (&sn)[8], float sign,
                                     bool interleaved, int partner)
{
    float o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float w = interleaved ? v[i ^ 1] : __shfl_sync(0xffffffffu, v[i], partner);
        o[i] = fmaf(v[i], cs[i], sign * sn[i] * w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = o[i];
}

template <int LANES> __device__ __forceinline__ float row_sum(float v)
{
#pragma unroll
    for (int m = LANES / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

template <typename T, int D, bool BACKWARD>
__global__ void __launch_bounds__(kThreads) head_norm_kernel(NormParams p)
{
    constexpr int LANES = D / 8, GROUPS = kThreads / LANES;
    const int lane = threadIdx.x & 31, l = lane % LANES, grp = threadIdx.x / LANES;
    // the lane that holds the partner channels of the half-split pairs (itself past R)
    const int hl = p.R / 16;
    const int partner = lane - l + (l < hl ? l + hl : l < 2 * hl ? l - hl : l);
    float acc[2][8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[0][i] = acc[1][i] = 0.f;
    const float scale = p.norm == 1 ? 1.f / D : 1.f;
    const int per_token = p.side[0].chunks + p.side[1].chunks;
    // a warp's groups run their loops together: shuffles need every lane
    const long long step = (long long)gridDim.x * GROUPS;
    const long long base = (long long)blockIdx.x * GROUPS + (threadIdx.x / 32) * (32 / LANES);
    for (long long task0 = base; task0 < p.tasks; task0 += step) {
        const long long task = task0 + grp % (32 / LANES);
        const bool ok = task < p.tasks;
        const long long token = ok ? task / per_token : 0;
        int chunk = ok ? (int)(task % per_token) : 0;
        const int sd = chunk >= p.side[0].chunks;
        if (sd) chunk -= p.side[0].chunks;
        const int H = sd ? p.side[1].H : p.side[0].H;
        const float *weight = sd ? p.side[1].weight : p.side[0].weight;
        const T *x = static_cast<const T *>(sd ? p.side[1].x : p.side[0].x) + token * (sd ? p.side[1].ld : p.side[0].ld) +
                     8 * l;
        const T *dy = static_cast<const T *>(sd ? p.side[1].dy : p.side[0].dy) + (size_t)token * H * D + 8 * l;
        T *out = static_cast<T *>(sd ? p.side[1].out : p.side[0].out) + (size_t)token * H * D + 8 * l;
        const int h0 = chunk * p.per, h1 = ok ? min(H, h0 + p.per) : h0;
        float cs[8], sn[8], w[8];
        if (ok) load_angles<D>(p, token, l, cs, sn);
        else
#pragma unroll
            for (int i = 0; i < 8; ++i) { cs[i] = 1.f; sn[i] = 0.f; }
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = weight ? __ldg(weight + 8 * l + i) : 1.f;
        for (int hh = 0; hh < p.per; hh += kHeads) {
            Raw<T, 8> rx[kHeads], ry[kHeads];
#pragma unroll
            for (int k = 0; k < kHeads; ++k) {
                const int h = h0 + hh + k;
                rx[k].zero();
                if (h < h1) rx[k].load_vec(x + (size_t)h * D);
                if constexpr (BACKWARD) {
                    ry[k].zero();
                    if (h < h1) ry[k].load_vec(dy + (size_t)h * D);
                }
            }
#pragma unroll
            for (int k = 0; k < kHeads; ++k) {
                const int h = h0 + hh + k;
                float v[8];
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) { v[i] = rx[k].get(i); ss = fmaf(v[i], v[i], ss); }
                float inv = 1.f;
                if (p.norm) {
                    ss = row_sum<LANES>(ss);
                    inv = rsqrtf(fmaf(ss, scale, p.eps));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= inv;
                if constexpr (!BACKWARD) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] *= w[i];
                    turn(v, cs, sn, 1.f, p.interleaved, partner);
                } else {
                    float g[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) g[i] = ry[k].get(i);
                    turn(g, cs, sn, -1.f, p.interleaved, partner);
                    float dot = 0.f;
                    const bool mine = h < h1;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float dw = mine ? g[i] * v[i] : 0.f;
                        acc[0][i] += sd ? 0.f : dw;
                        acc[1][i] += sd ? dw : 0.f;
                        g[i] *= w[i];
                        dot = fmaf(g[i], v[i], dot);
                    }
                    if (p.norm) dot = row_sum<LANES>(dot) * scale;
                    else dot = 0.f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = inv * fmaf(-v[i], dot, g[i]);
                }
                if (h < h1) store_vec<T, 8>(out + (size_t)h * D, v);
            }
        }
    }
    if constexpr (BACKWARD) {
        __shared__ float sm[GROUPS][2][D];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            sm[grp][0][8 * l + i] = acc[0][i];
            sm[grp][1][8 * l + i] = acc[1][i];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
            float s = 0.f;
            for (int k = 0; k < GROUPS; ++k) s += sm[k][i / D][i % D];
            p.part[(size_t)blockIdx.x * 2 * D + i] = s;
        }
    }
}

// dweight of both sides: one warp per value over the blocks' parts, always the same order.
__global__ void __launch_bounds__(256) head_norm_dweight_kernel(const float *part, int blocks, int d, float *dq, float *dk)
{
    const int lane = threadIdx.x & 31, i = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= 2 * d) return;
    float s = 0.f;
    for (int b = lane; b < blocks; b += 32) s += part[(size_t)b * 2 * d + i];
    s = row_sum<32>(s);
    float *out = i < d ? dq : dk;
    if (lane == 0 && out) out[i % d] = s;
}

int sm_count()
{
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

template <typename T, int D, bool BACKWARD>
cudaError_t launch(const HeadNormArgs &a, cudaStream_t st)
{
    constexpr int GROUPS = kThreads / (D / 8);
    const int sms = sm_count();
    NormParams p;
    // heads per task: all of a side where that still fills the GPU, else few, for latency
    const int most = a.side[0].H > a.side[1].H ? a.side[0].H : a.side[1].H;
    p.per = kHeads;
    while (p.per < most && a.tokens * ((most + 2 * p.per - 1) / (2 * p.per)) >= 8LL * sms * GROUPS) p.per *= 2;
    p.tokens = a.tokens;
    p.T = a.T > 0 ? a.T : 1;
    p.R = a.R; p.P = a.P; p.first = a.first;
    p.norm = a.norm; p.interleaved = a.interleaved; p.eps = a.eps;
    p.cos_sin = a.cos_sin; p.positions = a.positions;
    p.status = a.status;
    p.part = static_cast<float *>(a.workspace);
    int per_token = 0;
    for (int s = 0; s < 2; ++s) {
        const HeadNormSide &h = a.side[s];
        p.side[s] = Side{h.H, (h.H + p.per - 1) / p.per, h.x, h.dy, h.ld, h.weight, h.out};
        per_token += p.side[s].chunks;
    }
    p.tasks = a.tokens * per_token;
    const long long want = (p.tasks + GROUPS - 1) / GROUPS;
    const long long cap = BACKWARD ? (kMaxBlocks < 4LL * sms ? kMaxBlocks : 4LL * sms) : 16LL * sms;
    const int blocks = (int)(want < cap ? want : cap);
    if (blocks > 0) {
        head_norm_kernel<T, D, BACKWARD><<<blocks, kThreads, 0, st>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (BACKWARD && (a.side[0].dweight || a.side[1].dweight)) {
        head_norm_dweight_kernel<<<(2 * D + 7) / 8, 256, 0, st>>>(p.part, blocks, D, a.side[0].dweight, a.side[1].dweight);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

template <bool BACKWARD> cudaError_t dispatch(const HeadNormArgs &a, cudaStream_t st)
{
    if (a.bf16)
        return a.d == 64 ? launch<__nv_bfloat16, 64, BACKWARD>(a, st)
             : a.d == 128 ? launch<__nv_bfloat16, 128, BACKWARD>(a, st)
                          : launch<__nv_bfloat16, 256, BACKWARD>(a, st);
    return a.d == 64 ? launch<float, 64, BACKWARD>(a, st)
         : a.d == 128 ? launch<float, 128, BACKWARD>(a, st)
                      : launch<float, 256, BACKWARD>(a, st);
}

}  // namespace

size_t head_norm_backward_workspace_bytes(int d) { return (size_t)kMaxBlocks * 2 * d * sizeof(float); }
cudaError_t launch_head_norm_rope(const HeadNormArgs &a, cudaStream_t st) { return dispatch<false>(a, st); }
cudaError_t launch_head_norm_rope_backward(const HeadNormArgs &a, cudaStream_t st) { return dispatch<true>(a, st); }

}  // namespace gdr2
