// conv_backward.cu -- gradients of the block prologue's short convolution (prologue.cu):
// with u_t = sum_i w_i x_{t - (W-1) + i}, s = silu(u) and y = s, or y = s / r with
// r = sqrt(sum over the head of s^2 + eps),
//
//   ds = dy,  or  (dy - y (y . dy)) / r
//   du = ds silu'(u),  silu'(u) = sigma(u) (1 + u (1 - sigma(u)))
//   dx_t = sum_i w_i du_{t + (W-1) - i}  (+ the gradient of the final state, where t is one of its rows)
//   dw_i = sum_t du_t x_{t - (W-1) + i}
//
// A state before the sequence is its tokens -(W-1) .. -1, so its gradient is dx there.
//
// One pass over x and dy (u is formed again), one write of dx: an HBM stream of three
// tensors. A warp walks one head over a run of tokens with the last inputs and the unfinished
// dx rows in registers; it forms du for the W - 1 tokens after its run too, which its last dx
// rows need. The weights' gradient is summed in registers over the run, then over runs and
// sequences by a second kernel in a fixed order.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr2_launch.h"
#include "seq_ops.h"

namespace gdr2 {
namespace {

using namespace seq;

constexpr int kMaxWidth = 4;
constexpr int kRun = 64;   // tokens per warp task
constexpr int kWarps = 8;
constexpr int kAhead = 4;  // tokens whose loads are in flight

struct ConvBwdParams {
    int N, T, H, W, runs;
    float eps;
    const void *x, *dy, *sin, *dsout;
    const float *weight;
    void *dx, *dsin;
    float *part;  // [N runs][H d][kMaxWidth]
};

template <typename T, int D, bool L2>
__global__ void __launch_bounds__(kWarps * 32) conv_backward_kernel(ConvBwdParams p)
{
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long task = (long long)blockIdx.x * kWarps + warp;
    if (task >= (long long)p.N * p.H * p.runs) return;
    const int h = (int)(task % p.H);
    const long long nr = task / p.H;  // sequence and run
    const int run = (int)(nr % p.runs), n = (int)(nr / p.runs);
    const int t0 = run * kRun, t1 = min(p.T, t0 + kRun);
    const size_t HD = (size_t)p.H * D, col = (size_t)h * D + lane * V;
    const T *x = static_cast<const T *>(p.x) + (size_t)n * p.T * HD + col;
    const T *dy = static_cast<const T *>(p.dy) + (size_t)n * p.T * HD + col;
    T *dx = static_cast<T *>(p.dx) + (size_t)n * p.T * HD + col;
    const size_t srow = (size_t)n * (p.W - 1);

    float wt[kMaxWidth][V];  // right-aligned: wt[i] multiplies the input kMaxWidth - 1 - i back
#pragma unroll
    for (int i = 0; i < kMaxWidth; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int j = i - (kMaxWidth - p.W);
            wt[i][v] = j >= 0 ? __ldg(p.weight + (col + v) * p.W + j) : 0.f;
        }
    float xw[kMaxWidth][V], dxp[kMaxWidth][V], dw[kMaxWidth][V];
#pragma unroll
    for (int i = 0; i < kMaxWidth; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) xw[i][v] = dxp[i][v] = dw[i][v] = 0.f;
    // xw[i + 1] = input t0 - 3 + i: a token, a state row or zero
#pragma unroll
    for (int i = 0; i < kMaxWidth - 1; ++i) {
        const int t = t0 - (kMaxWidth - 1) + i, js = t + p.W - 1;
        Raw<T, V> r;
        r.zero();
        if (t >= 0) r.load_vec(x + (size_t)t * HD);
        else if (p.sin && js >= 0) r.load_vec(static_cast<const T *>(p.sin) + (srow + js) * HD + col);
#pragma unroll
        for (int v = 0; v < V; ++v) xw[i + 1][v] = r.get(v);
    }
    Raw<T, V> nx[kAhead], ny[kAhead];
    auto fetch = [&](int j0) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            nx[k].zero();
            ny[k].zero();
            if (j0 + k < p.T && j0 + k < t1 + kMaxWidth - 1) {
                nx[k].load_vec(x + (size_t)(j0 + k) * HD);
                ny[k].load_vec(dy + (size_t)(j0 + k) * HD);
            }
        }
    };
    const int jend = t1 + kMaxWidth - 1, first = t0 == 0 ? -(p.W - 1) : t0;
    fetch(t0);
    for (int j0 = t0; j0 < jend; j0 += kAhead) {
        Raw<T, V> cx[kAhead], cy[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) { cx[k] = nx[k]; cy[k] = ny[k]; }
        fetch(j0 + kAhead);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int j = j0 + k;
            if (j >= jend) break;
            float y[V], ds[V], du[V], sg[V], u[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int i = 0; i < kMaxWidth - 1; ++i) xw[i][v] = xw[i + 1][v];
                xw[kMaxWidth - 1][v] = cx[k].get(v);
                float a = 0.f;
#pragma unroll
                for (int i = 0; i < kMaxWidth; ++i) a = fmaf(wt[i][v], xw[i][v], a);
                u[v] = a;
                sg[v] = sigmoid(a);
                y[v] = a * sg[v];
                ds[v] = cy[k].get(v);  // zero past the sequence: its du is zero
            }
            if constexpr (L2) {
                float ss = 0.f, dot = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    ss = fmaf(y[v], y[v], ss);
                    dot = fmaf(y[v], ds[v], dot);
                }
#pragma unroll
                for (int m = 16; m >= 1; m >>= 1) {
                    ss += __shfl_xor_sync(0xffffffffu, ss, m);
                    dot += __shfl_xor_sync(0xffffffffu, dot, m);
                }
                const float inv = j < p.T ? rsqrtf(ss + p.eps) : 0.f;
                const float f = dot * inv * inv;
#pragma unroll
                for (int v = 0; v < V; ++v) ds[v] = inv * fmaf(-y[v], f, ds[v]);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                du[v] = ds[v] * sg[v] * fmaf(u[v], 1.f - sg[v], 1.f);
                if (j >= p.T) du[v] = 0.f;
                if (j < t1)
#pragma unroll
                    for (int i = 0; i < kMaxWidth; ++i) dw[i][v] = fmaf(du[v], xw[i][v], dw[i][v]);
#pragma unroll
                for (int i = 0; i < kMaxWidth; ++i) dxp[i][v] = fmaf(wt[i][v], du[v], dxp[i][v]);
            }
            // dxp[i] belongs to token j - 3 + i: the first is finished
            const int t = j - (kMaxWidth - 1);
            if (t >= first && t < t1) {
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) o[v] = dxp[0][v];
                const int js = t - (p.T - (p.W - 1));  // the final state's row that holds this input
                if (p.dsout && js >= 0) {
                    Raw<T, V> r;
                    r.load_vec(static_cast<const T *>(p.dsout) + (srow + js) * HD + col);
#pragma unroll
                    for (int v = 0; v < V; ++v) o[v] += r.get(v);
                }
                if (t >= 0) store_vec<T, V>(dx + (size_t)t * HD, o);
                else if (p.dsin) store_vec<T, V>(static_cast<T *>(p.dsin) + (srow + t + p.W - 1) * HD + col, o);
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
#pragma unroll
                for (int i = 0; i < kMaxWidth - 1; ++i) dxp[i][v] = dxp[i + 1][v];
                dxp[kMaxWidth - 1][v] = 0.f;
            }
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v)
        *reinterpret_cast<float4 *>(p.part + ((size_t)nr * HD + col + v) * kMaxWidth) =
            make_float4(dw[0][v], dw[1][v], dw[2][v], dw[3][v]);
}

// dweight: the runs' parts, eight groups of them summed side by side and then in order.
__global__ void __launch_bounds__(256) conv_dweight_kernel(const float *part, long long parts, long long values, int W,
                                                           float *dweight)
{
    __shared__ float sm[8][32];
    const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const long long i = (long long)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (i < values)
#pragma unroll 8
        for (long long k = grp; k < parts; k += 8) s += part[k * values + i];
    sm[grp][lane] = s;
    __syncthreads();
    if (grp == 0 && i < values) {
        float a = 0.f;
#pragma unroll
        for (int k = 0; k < 8; ++k) a += sm[k][lane];
        const int j = (int)(i % kMaxWidth) - (kMaxWidth - W);
        if (j >= 0) dweight[i / kMaxWidth * W + j] = a;
    }
}

template <typename T, int D>
cudaError_t launch(const ConvBwdParams &p, bool l2, float *dweight, cudaStream_t st)
{
    const long long tasks = (long long)p.N * p.H * p.runs;
    const unsigned blocks = (unsigned)((tasks + kWarps - 1) / kWarps);
    if (l2) conv_backward_kernel<T, D, true><<<blocks, kWarps * 32, 0, st>>>(p);
    else conv_backward_kernel<T, D, false><<<blocks, kWarps * 32, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long values = (long long)p.H * D * kMaxWidth;
    conv_dweight_kernel<<<(unsigned)((values + 31) / 32), 256, 0, st>>>(p.part, (long long)p.N * p.runs, values, p.W,
                                                                       dweight);
    return cudaGetLastError();
}

int runs_of(int T) { return T > 0 ? (T + kRun - 1) / kRun : 1; }

}  // namespace

size_t conv_backward_workspace_bytes(int N, int T, int H, int d)
{
    return ((size_t)N * runs_of(T) * H * d * kMaxWidth * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_conv_backward(const ConvBwdArgs &a, cudaStream_t st)
{
    ConvBwdParams p;
    p.N = a.N; p.T = a.T; p.H = a.H; p.W = a.width;
    p.runs = runs_of(a.T);
    p.eps = a.eps;
    p.x = a.x; p.dy = a.dy; p.sin = a.state_in; p.dsout = a.dstate_out;
    p.weight = a.weight;
    p.dx = a.dx; p.dsin = a.dstate_in;
    p.part = static_cast<float *>(a.workspace);
    if (a.bf16)
        return a.d == 128 ? launch<__nv_bfloat16, 128>(p, a.l2norm, a.dweight, st)
                          : launch<__nv_bfloat16, 64>(p, a.l2norm, a.dweight, st);
    return a.d == 128 ? launch<float, 128>(p, a.l2norm, a.dweight, st) : launch<float, 64>(p, a.l2norm, a.dweight, st);
}

}  // namespace gdr2
