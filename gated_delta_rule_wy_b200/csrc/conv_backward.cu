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
// tensors. A warp walks one head over a run of tokens, four loads in flight. Of two tokens at a time the head's
// two sums are taken by one butterfly that halves the four values with each step (10 shuffles instead of 20);
// the last inputs and the unfinished dx rows stay in registers, pairs of channels in one 64-bit register each. It
// forms du for the W - 1 tokens after its run too, which its last dx rows need. The weights' gradient is summed in registers over the run, then over runs and
// sequences by a second kernel in a fixed order.
//
// What bounds it: 34 instructions per element, at half an instruction per cycle from 12 warps: 68 us for 4 x 4096
// tokens of 16 heads of 128 channels in bf16 with the norm (3.0 TB/s; the three tensors' HBM time is 31 us).

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "gdr2_launch.h"
#include "seq_ops.h"

namespace gdr2 {
namespace {

using namespace seq;

constexpr int kMaxWidth = 4;
constexpr int kWarps = 4;
constexpr int kBatch = 4;  // tokens at a time: the width's ring of unfinished rows is back in place after four
// Blocks per SM that the registers are held to. (bf16, 4 x 4096 tokens of 16 heads: d = 128 with the norm 68 us at three, 92
// at four with spills, 78 at two; without it 63 at three, 55 to 64 at four; d = 64 with the norm 44 at four, 50 at three.)
template <int D> constexpr int blocks_per_sm() { return D == 64 ? 4 : 3; }
static_assert(kBatch == kMaxWidth, "a batch turns the ring once");

struct ConvBwdParams {
    int N, T, H, W, run, runs;  // run: tokens per warp task (a multiple of kBatch)
    float eps;
    const void *x, *dy, *sin, *dsout;
    const float *weight;
    void *dx, *dsin;
    float *part;  // [N runs][H d][kMaxWidth]
};

// The pairs of V elements of one row, and back
template <typename T, int V> __device__ __forceinline__ void to_pairs(const Raw<T, V> &r, f32x2 (&v)[V / 2])
{
#pragma unroll
    for (int i = 0; i < V / 2; ++i) v[i] = pair(r.get(2 * i), r.get(2 * i + 1));
}
template <typename T, int V> __device__ __forceinline__ void store_pairs(T *p, const f32x2 (&v)[V / 2])
{
    float o[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) split(v[i], o[2 * i], o[2 * i + 1]);
    store_vec<T, V>(p, o);
}

// Sums of four values over a warp, in every lane.
__device__ __forceinline__ void warp_sums(float (&v)[4], int lane)
{
    constexpr unsigned all = 0xffffffffu;
#pragma unroll
    for (int w = 2, m = 16; w >= 1; w /= 2, m /= 2) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < w; ++i)
            v[i] = (up ? v[i + w] : v[i]) + __shfl_xor_sync(all, up ? v[i] : v[i + w], m);
    }
    float s = v[0];  // of value lane / 8
#pragma unroll
    for (int m = 4; m >= 1; m /= 2) s += __shfl_xor_sync(all, s, m);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(all, s, 8 * i);
}

// FULL: all kMaxWidth taps. With fewer the missing ones are skipped, not multiplied by zero: an infinite input
// reaches no row beyond the width.
template <typename T, int D, bool L2, bool FULL>
__global__ void __launch_bounds__(kWarps * 32, blocks_per_sm<D>()) conv_backward_kernel(ConvBwdParams p)
{
    constexpr int V = D / 32, P = V / 2, kLast = kMaxWidth - 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long task = (long long)blockIdx.x * kWarps + warp;
    if (task >= (long long)p.N * p.H * p.runs) return;
    const int h = (int)(task % p.H);
    const long long nr = task / p.H;  // sequence and run
    const int run = (int)(nr % p.runs), n = (int)(nr / p.runs);
    const int t0 = run * p.run, t1 = min(p.T, t0 + p.run);
    const size_t HD = (size_t)p.H * D, col = (size_t)h * D + lane * V;
    const T *x = static_cast<const T *>(p.x) + (size_t)n * p.T * HD + col;
    const T *dy = static_cast<const T *>(p.dy) + (size_t)n * p.T * HD + col;
    T *dx = static_cast<T *>(p.dx) + (size_t)n * p.T * HD + col;
    const size_t srow = (size_t)n * (p.W - 1);
    const int skip = FULL ? 0 : kMaxWidth - p.W;

    f32x2 wt[kMaxWidth][P];  // right-aligned: wt[i] multiplies the input kLast - i back
#pragma unroll
    for (int i = 0; i < kMaxWidth; ++i)
#pragma unroll
        for (int v = 0; v < P; ++v) {
            const int j = i - (kMaxWidth - p.W);
            wt[i][v] = j >= 0 ? pair(__ldg(p.weight + (col + 2 * v) * p.W + j), __ldg(p.weight + (col + 2 * v + 1) * p.W + j))
                              : 0;
        }
    // xw[i]: input j0 - kLast + i of the batch at j0; dxp: ring of the unfinished rows, token j in slot (j - t0 + 3) % 4
    f32x2 xw[kLast + kBatch][P], dxp[kMaxWidth][P], dw[kMaxWidth][P];
#pragma unroll
    for (int i = 0; i < kMaxWidth; ++i)
#pragma unroll
        for (int v = 0; v < P; ++v) dxp[i][v] = dw[i][v] = 0;
#pragma unroll
    for (int i = 0; i < kLast; ++i) {  // a token, a state row or zero
        const int t = t0 - kLast + i, js = t + p.W - 1;
        Raw<T, V> r;
        r.zero();
        if (t >= 0 && t < p.T) r.load_vec(x + (size_t)t * HD);
        else if (t < 0 && p.sin && js >= 0) r.load_vec(static_cast<const T *>(p.sin) + (srow + js) * HD + col);
        to_pairs<T, V>(r, xw[i]);
    }
    const f32x2 one = pair(1.f, 1.f), minus = pair(-1.f, -1.f);
    // tokens past the sequence read its last one, and are cleared when they are used
    Raw<T, V> nx[kBatch], ny[kBatch];
    auto fetch = [&](int j0) {
        if (j0 + kBatch <= p.T) {
            const T *px = x + (size_t)j0 * HD, *py = dy + (size_t)j0 * HD;
#pragma unroll
            for (int k = 0; k < kBatch; ++k, px += HD, py += HD) {
                nx[k].load_vec(px);
                ny[k].load_vec(py);
            }
            return;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const size_t at = (size_t)min(j0 + k, p.T - 1) * HD;
            nx[k].load_vec(x + at);
            ny[k].load_vec(dy + at);
        }
    };
    const int jend = t1 + kLast, first = t0 == 0 ? -(p.W - 1) : t0;
    if (p.T > 0) fetch(t0);
    else
#pragma unroll
        for (int k = 0; k < kBatch; ++k) { nx[k].zero(); ny[k].zero(); }
    f32x2 u[2][P], sg[2][P], g[2][P];
    float inv[2], f[2];
    // INNER: every token of the batch is one of the run's, and every row it finishes is one of the run's tokens
    // that no final state holds: none of the tests below
    auto batch = [&](int j0, auto inner) {
        constexpr bool INNER = decltype(inner)::value;
        T *out = dx + (size_t)(INNER ? j0 - kLast : 0) * HD;
        if (!INNER && j0 + kBatch > p.T)
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (j0 + k >= p.T) { nx[k].zero(); ny[k].zero(); }
        Raw<T, V> gy[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            to_pairs<T, V>(nx[k], xw[kLast + k]);
            gy[k] = ny[k];
        }
        if (j0 + kBatch < jend && p.T > 0) fetch(j0 + kBatch);
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            // two tokens' sums are taken together
            constexpr int kSub = 2;
            if (k % kSub == 0) {
                [[maybe_unused]] float sums[2 * kSub];
#pragma unroll
                for (int b = 0; b < kSub; ++b) {
                    [[maybe_unused]] f32x2 ss = 0, dot = 0;
                    to_pairs<T, V>(gy[k + b], g[b]);
#pragma unroll
                    for (int v = 0; v < P; ++v) {
                        f32x2 a = mul2(wt[kLast][v], xw[k + b + kLast][v]);
#pragma unroll
                        for (int i = kLast - 1; i >= 0; --i)
                            if (i >= skip) a = fma2(wt[i][v], xw[k + b + i][v], a);
                        float lo, hi;
                        split(a, lo, hi);
                        u[b][v] = a;
                        sg[b][v] = pair(sigmoid(lo), sigmoid(hi));
                        if constexpr (L2) {
                            const f32x2 y = mul2(a, sg[b][v]);
                            ss = v ? fma2(y, y, ss) : mul2(y, y);
                            dot = v ? fma2(y, g[b][v], dot) : mul2(y, g[b][v]);
                        }
                    }
                    if constexpr (L2) {
                        float lo, hi;
                        split(ss, lo, hi);
                        sums[2 * b] = lo + hi;
                        split(dot, lo, hi);
                        sums[2 * b + 1] = lo + hi;
                    }
                }
                if constexpr (L2) {
                    warp_sums(sums, lane);
#pragma unroll
                    for (int b = 0; b < kSub; ++b) {
                        // past the sequence nothing is left of dy, but eps = 0 would leave 0 / 0
                        inv[b] = INNER || j0 + k + b < p.T ? rsqrtf(sums[2 * b] + p.eps) : 0.f;
                        f[b] = -sums[2 * b + 1] * inv[b] * inv[b];
                    }
                }
            }
            const int j = j0 + k, b = k % kSub;
            f32x2 du[P];
#pragma unroll
            for (int v = 0; v < P; ++v) {
                const f32x2 s = sg[b][v], slope = mul2(s, fma2(u[b][v], fma2(minus, s, one), one));
                f32x2 ds = g[b][v];
                if constexpr (L2) ds = mul2(pair(inv[b], inv[b]), fma2(mul2(u[b][v], s), pair(f[b], f[b]), ds));
                du[v] = mul2(ds, slope);
            }
            if (!INNER && j >= p.T)  // (its slope may be that of an infinite window)
#pragma unroll
                for (int v = 0; v < P; ++v) du[v] = 0;
            if (INNER || j < t1)
#pragma unroll
                for (int v = 0; v < P; ++v)
#pragma unroll
                    for (int i = 0; i < kMaxWidth; ++i)
                        if (i >= skip) dw[i][v] = fma2(du[v], xw[k + i][v], dw[i][v]);
#pragma unroll
            for (int v = 0; v < P; ++v)
#pragma unroll
                for (int i = 0; i < kMaxWidth; ++i) {
                    if (i == kLast) dxp[(k + i) % 4][v] = mul2(wt[i][v], du[v]);
                    else if (i >= skip) dxp[(k + i) % 4][v] = fma2(wt[i][v], du[v], dxp[(k + i) % 4][v]);
                }
            const int t = j - kLast;  // its row is finished
            if constexpr (INNER) {
                store_pairs<T, V>(out, dxp[k]);
                out += HD;
            } else if (t >= first && t < t1) {
                const int js = t - (p.T - (p.W - 1));  // the final state's row that holds this input
                if (p.dsout && js >= 0) {
                    Raw<T, V> r;
                    f32x2 d[P];
                    r.load_vec(static_cast<const T *>(p.dsout) + (srow + js) * HD + col);
                    to_pairs<T, V>(r, d);
#pragma unroll
                    for (int v = 0; v < P; ++v) dxp[k][v] = add2(dxp[k][v], d[v]);
                }
                if (t >= 0) store_pairs<T, V>(dx + (size_t)t * HD, dxp[k]);
                else if (p.dsin) store_pairs<T, V>(static_cast<T *>(p.dsin) + (srow + t + p.W - 1) * HD + col, dxp[k]);
            }
        }
#pragma unroll
        for (int i = 0; i < kLast; ++i)
#pragma unroll
            for (int v = 0; v < P; ++v) xw[i][v] = xw[kBatch + i][v];
    };
    for (int j0 = t0; j0 < jend; j0 += kBatch) {
        if (j0 >= t0 + kLast && j0 + kBatch <= t1) batch(j0, std::true_type{});
        else batch(j0, std::false_type{});
    }
#pragma unroll
    for (int v = 0; v < P; ++v) {
        float4 a, b;
        split(dw[0][v], a.x, b.x);
        split(dw[1][v], a.y, b.y);
        split(dw[2][v], a.z, b.z);
        split(dw[3][v], a.w, b.w);
        float4 *o = reinterpret_cast<float4 *>(p.part + ((size_t)nr * HD + col + 2 * v) * kMaxWidth);
        o[0] = a;
        o[1] = b;
    }
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
    const bool full = p.W == kMaxWidth;
    auto *kern = l2 ? full ? conv_backward_kernel<T, D, true, true> : conv_backward_kernel<T, D, true, false>
                    : full ? conv_backward_kernel<T, D, false, true> : conv_backward_kernel<T, D, false, false>;
    kern<<<blocks, kWarps * 32, 0, st>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long values = (long long)p.H * D * kMaxWidth;
    conv_dweight_kernel<<<(unsigned)((values + 31) / 32), 256, 0, st>>>(p.part, (long long)p.N * p.runs, values, p.W,
                                                                       dweight);
    return cudaGetLastError();
}

// Tokens per warp task: every run costs its tokens, the kLast after them and a start, and the GPU runs a number of
// tasks at once; few sequences are cut short for latency, many run longer.
int run_of(int N, int T, int H, int d)
{
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const long long slots = (long long)(sms > 0 ? sms : 148) * (d == 64 ? blocks_per_sm<64>() : blocks_per_sm<128>()) * kWarps;
    int best = 8;
    long long least = -1;
    for (int run = 8; run <= 256; run += run < 32 ? 4 : 16) {
        const long long tasks = (long long)N * H * ((T + run - 1) / run);
        const long long cost = (tasks + slots - 1) / slots * (run + 12);
        if (least < 0 || cost < least) { least = cost; best = run; }
    }
    return best;
}
int runs_of(int T, int run) { return T > 0 ? (T + run - 1) / run : 1; }

}  // namespace

size_t conv_backward_workspace_bytes(int N, int T, int H, int d)
{
    return ((size_t)N * runs_of(T, run_of(N, T, H, d)) * H * d * kMaxWidth * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_conv_backward(const ConvBwdArgs &a, cudaStream_t st)
{
    ConvBwdParams p;
    p.N = a.N; p.T = a.T; p.H = a.H; p.W = a.width;
    p.run = run_of(a.N, a.T, a.H, a.d);
    p.runs = runs_of(a.T, p.run);
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
