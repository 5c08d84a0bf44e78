// ssm_backward.cu -- gradients of the selective state-space scan (ssm_scan.cu), dense
// sequences. With g = dy silu(z) and a_t = exp(D_t A), the gradient of the state obeys the
// same recurrence from the last token to the first,
//
//   dh_t = C_t g_t + a_{t+1} dh_{t+1}                (plus dS_T at the last token)
//   dC_t[n] = sum_c g_t h_t,   dB_t[n] = sum_c D_t x_t dh_t,   du_t = sum_n B_t[n] dh_t
//   m_t = dh_t a_t h_{t-1}  (the gradient of the exponent D_t A)
//   dx_t = D_t du_t + Dskip g_t,   dD_t = x_t du_t + sum_n A m_t,   ddt = dD softplus'
//   dA = sum_t D_t m_t,  dDskip = sum g x,  dbias = sum ddt,  dS0 = a_0 dh_0
//   dz_t = dy_t y'_t silu'(z_t) with y' the output before its gate, formed again here.
//
// The states are formed again from the ones saved every kSsmChunk tokens: per chunk a thread
// runs its four states forward and keeps them in registers (64 of them), then walks back.
// The two sums over channels (dB, dC) are taken over a warp's channels by shuffles that halve
// the values with each step, over a block's warps in shared memory and over the blocks by a
// last kernel, in a fixed order: no atomics, the same bits each time.
//
// Segments of the time axis as in the forward: each segment's own part of the gradient that
// leaves it to the left and the sum of its step sizes, then every segment from the
// composition of those to its right.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "gdr2_launch.h"
#include "seq_ops.h"

namespace gdr2 {
namespace {

using namespace seq;

constexpr int kThreads = 256;
constexpr int kTile = kSsmChunk;

struct BwdParams {
    int B, T, D, seg, nseg, nchunk, ncb;
    bool softplus;
    const void *x, *dt, *z, *Bm, *Cm, *dy;
    long long ldx, lddt, ldz, ldb, ldc;
    const float *A, *Dskip, *bias, *dS_T, *saved;
    void *dx, *ddt, *dz;
    float *dS0;
    float *eloc, *dsum;      // [B][nseg][D][N], [B][nseg][D]
    float *pBC;              // [ncb][B T][2 N] sums over one block's channels of dB, dC
    float *pA;               // [B nseg][D][N] sums over one segment of dA
    float *pD;               // [B nseg][2][D] of dDskip, dbias
};

template <int N> struct BwdShape {
    static constexpr int L = N / 4;
    static constexpr int CH = kThreads / L;
    static constexpr int E = CH / 16 < 2 ? 2 : CH / 16;  // channels a thread loads of one token
    static constexpr int kPerRow = CH / E;               // threads per token (16; 8 at N = 64)
    static constexpr int kPad = 8;
    static constexpr int kRow = CH + kPad;
    static constexpr int kWarps = kThreads / 32;
    // shared memory, in floats: (D, D x) then (du, sum A m); g; y before its gate; B; C; the warps' sums
    static constexpr int kDx = 0, kG = 2 * kTile * kRow, kY = kG + kTile * kRow, kB = kY + kTile * kRow;
    static constexpr int kC = kB + kTile * N, kRed = kC + kTile * N, kFloats = kRed + kWarps * kTile * 2 * N;
};

// Sum over a warp's 32 / L channels (lane bits log2 L .. 4) of eight values per lane, which
// halve with each step; lane (channel bits j) ends with value(s) index0 ...; returns how many.
template <int L> struct ChannelSum {
    static constexpr int kLeft = L == 2 ? 1 : L == 4 ? 1 : L == 8 ? 2 : 4;  // values per lane at the end
    __device__ __forceinline__ static void run(float (&v)[8], int lane, int &index)
    {
        index = 0;
        int width = 8;
#pragma unroll
        for (int m = L; m < 32; m <<= 1) {
            if (width > 1) {
                const bool up = lane & m;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i < width / 2) {
                        const float keep = up ? v[i + width / 2] : v[i];
                        const float give = up ? v[i] : v[i + width / 2];
                        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
                    }
                }
                width /= 2;
                index += up ? width : 0;
            } else {
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], m);
            }
        }
    }
};

template <int L> __device__ __forceinline__ float lane_sum(float v)
{
#pragma unroll
    for (int m = 1; m < L; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// SUMMARY: the segment's own part of the gradient that leaves it to the left, and sum D.
template <typename T, int N, bool VEC, bool SUMMARY>
__global__ void __launch_bounds__(kThreads) ssm_backward_kernel(BwdParams p)
{
    using S = BwdShape<N>;
    constexpr int L = S::L, CH = S::CH, E = S::E, kRow = S::kRow;
    constexpr int kBC = (kTile * N + kThreads - 1) / kThreads;
    extern __shared__ __align__(16) float smem[];
    float2 *sdx = reinterpret_cast<float2 *>(smem + S::kDx);
    float *sg = smem + S::kG, *sy = smem + S::kY, *sB = smem + S::kB, *sC = smem + S::kC, *sred = smem + S::kRed;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int stream = blockIdx.x / p.ncb, cb = blockIdx.x % p.ncb;
    const int g = SUMMARY ? blockIdx.y + 1 : blockIdx.y;
    const int c0 = cb * CH;
    const int tbeg = g * p.seg, tend = min(p.T, tbeg + p.seg);
    const int ch = tid / L, q = tid % L, c = c0 + ch;
    const bool live = c < p.D;
    const int lr = tid / S::kPerRow, lc = (tid % S::kPerRow) * E;
    const int lvalid = lr < kTile ? min(E, p.D - (c0 + lc)) : 0;

    float A[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
        const float4 a = *reinterpret_cast<const float4 *>(p.A + (size_t)c * N + 4 * q);
        A[0] = a.x; A[1] = a.y; A[2] = a.z; A[3] = a.w;
    }
    float A2[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) A2[k] = A[k] * kLog2e;
    auto load_state = [&](const float *base, size_t index, float (&v)[4]) {
        const float4 a = *reinterpret_cast<const float4 *>(base + (index * p.D + c) * N + 4 * q);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    };
    auto store_state = [&](float *base, size_t index, const float (&v)[4]) {
        *reinterpret_cast<float4 *>(base + (index * p.D + c) * N + 4 * q) = make_float4(v[0], v[1], v[2], v[3]);
    };
    // e = a_{t+1} dh_{t+1}, the gradient that enters this segment from the right
    if (live) {
        if (g == p.nseg - 1) {
            if (p.dS_T) load_state(p.dS_T, stream, e);
        } else if (!SUMMARY) {
            load_state(p.eloc, (size_t)stream * p.nseg + p.nseg - 1, e);
            for (int i = p.nseg - 2; i > g; --i) {
                const size_t at = (size_t)stream * p.nseg + i;
                const float ds = p.dsum[at * p.D + c];
                float o[4];
                load_state(p.eloc, at, o);
#pragma unroll
                for (int k = 0; k < 4; ++k) e[k] = fmaf(ex2(ds * A2[k]), e[k], o[k]);
            }
        }
    }
    float bias[E], skip[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = p.bias && i < lvalid ? __ldg(p.bias + c0 + lc + i) : 0.f;
        skip[i] = p.Dskip && i < lvalid ? __ldg(p.Dskip + c0 + lc + i) : 0.f;
    }
    const T *x = static_cast<const T *>(p.x), *dt = static_cast<const T *>(p.dt), *z = static_cast<const T *>(p.z);
    const T *dy = static_cast<const T *>(p.dy);
    const T *Bm = static_cast<const T *>(p.Bm), *Cm = static_cast<const T *>(p.Cm);
    auto load_run = [&](const T *base, long long ld, int t, Raw<T, E> &r) {
        if (t >= tend || lvalid <= 0) { r.zero(); return; }
        const T *src = base + ((size_t)stream * p.T + t) * ld + c0 + lc;
        if constexpr (VEC) r.load_vec(src);
        else r.load_each(src, lvalid);
    };
    auto store_run = [&](void *base, int t, const float (&v)[E]) {
        T *dst = static_cast<T *>(base) + ((size_t)stream * p.T + t) * p.D + c0 + lc;
        if constexpr (VEC) store_vec<T, E>(dst, v);
        else store_each<T, E>(dst, v, lvalid);
    };
    Raw<T, E> rx, rdt, rz, rdy, nx, ndt, nz, ndy;
    float nb[kBC], nc[kBC];
    auto fetch = [&](int t0) {
        load_run(x, p.ldx, t0 + lr, nx);
        load_run(dt, p.lddt, t0 + lr, ndt);
        load_run(dy, p.D, t0 + lr, ndy);
        if (z) load_run(z, p.ldz, t0 + lr, nz);
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            const int r = (tid + i * kThreads) / N, n = (tid + i * kThreads) % N, t = t0 + r;
            const size_t row = (size_t)stream * p.T + t;
            nb[i] = r < kTile && t < tend ? load_one(Bm + row * p.ldb + n) : 0.f;
            nc[i] = r < kTile && t < tend ? load_one(Cm + row * p.ldc + n) : 0.f;
        }
    };
    float dA[4] = {0.f, 0.f, 0.f, 0.f}, dsum = 0.f;
    float aD[E], ab[E];
#pragma unroll
    for (int i = 0; i < E; ++i) aD[i] = ab[i] = 0.f;
    const int nt = (tend - tbeg + kTile - 1) / kTile;
    fetch(tbeg + (nt - 1) * kTile);
    for (int it = nt - 1; it >= 0; --it) {
        const int t0 = tbeg + it * kTile;
        rx = nx; rdt = ndt; rz = nz; rdy = ndy;
        const bool run_ok = t0 + lr < tend && lvalid > 0;
#pragma unroll
        for (int i = 0; i < E && lr < kTile; ++i) {
            const float v = rdt.get(i) + bias[i];
            const float d = run_ok && i < lvalid ? (p.softplus ? softplus(v) : v) : 0.f;
            float gv = rdy.get(i);
            if (z) { const float zv = rz.get(i); gv *= zv * sigmoid(zv); }
            sdx[lr * kRow + lc + i] = make_float2(d, d * rx.get(i));
            sg[lr * kRow + lc + i] = gv;  // zero past the segment and past D (dy was filled with zeros)
        }
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            const int at = tid + i * kThreads;
            if (at < kTile * N) { sB[at] = nb[i]; sC[at] = nc[i]; }
        }
        __syncthreads();
        if (it > 0) fetch(t0 - kTile);
        if constexpr (SUMMARY) {
#pragma unroll
            for (int t = kTile - 1; t >= 0; --t) {
                const float d = sdx[t * kRow + ch].x, gv = sg[t * kRow + ch];
                const float4 cv = *reinterpret_cast<const float4 *>(sC + t * N + 4 * q);
                dsum += d;
                e[0] = ex2(d * A2[0]) * fmaf(cv.x, gv, e[0]);
                e[1] = ex2(d * A2[1]) * fmaf(cv.y, gv, e[1]);
                e[2] = ex2(d * A2[2]) * fmaf(cv.z, gv, e[2]);
                e[3] = ex2(d * A2[3]) * fmaf(cv.w, gv, e[3]);
            }
            __syncthreads();
        } else {
            float h0[4] = {0.f, 0.f, 0.f, 0.f}, hist[kTile][4];
            if (live) load_state(p.saved, (size_t)stream * p.nchunk + t0 / kTile, h0);
#pragma unroll
            for (int t = 0; t < kTile; ++t) {
                const float2 dx = sdx[t * kRow + ch];
                const float4 b = *reinterpret_cast<const float4 *>(sB + t * N + 4 * q);
                const float bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float prev = t ? hist[t ? t - 1 : 0][k] : h0[k];
                    hist[t][k] = fmaf(ex2(dx.x * A2[k]), prev, dx.y * bb[k]);
                }
            }
#pragma unroll
            for (int t = kTile - 1; t >= 0; --t) {
                const float2 dx = sdx[t * kRow + ch];
                const float gv = sg[t * kRow + ch];
                const float4 b = *reinterpret_cast<const float4 *>(sB + t * N + 4 * q);
                const float4 cv = *reinterpret_cast<const float4 *>(sC + t * N + 4 * q);
                const float bb[4] = {b.x, b.y, b.z, b.w}, cc[4] = {cv.x, cv.y, cv.z, cv.w};
                float v[8], du = 0.f, dd = 0.f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float prev = t ? hist[t ? t - 1 : 0][k] : h0[k];
                    const float a = ex2(dx.x * A2[k]);
                    const float dh = fmaf(cc[k], gv, e[k]);
                    v[k] = dx.y * dh;
                    v[4 + k] = gv * hist[t][k];
                    du = fmaf(bb[k], dh, du);
                    e[k] = a * dh;
                    const float m = e[k] * prev;
                    dd = fmaf(A[k], m, dd);
                    dA[k] = fmaf(dx.x, m, dA[k]);
                }
                du = lane_sum<L>(du);
                dd = lane_sum<L>(dd);
                if (q == 0) sdx[t * kRow + ch] = make_float2(du, dd);  // after every lane's reads of this slot
                if (z) {
                    float yv = fmaf(cc[0], hist[t][0], cc[1] * hist[t][1]) + fmaf(cc[2], hist[t][2], cc[3] * hist[t][3]);
                    yv = lane_sum<L>(yv);
                    if (q == 0) sy[t * kRow + ch] = yv;
                }
                int at;
                ChannelSum<L>::run(v, lane, at);
                // value index j of a lane: j < 4 is dB of state 4 q + j, else dC of 4 q + j - 4
                if (L > 2 || lane < 16)
#pragma unroll
                    for (int i = 0; i < ChannelSum<L>::kLeft; ++i) {
                        const int j = at + i;
                        sred[(warp * kTile + t) * 2 * N + (j < 4 ? 0 : N) + 4 * q + (j & 3)] = v[i];
                    }
            }
            __syncthreads();
            if (run_ok) {
                float odx[E], odt[E], oz[E];
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    const int at = lr * kRow + lc + i;
                    const float2 s = sdx[at];
                    const float v = rdt.get(i) + bias[i], xv = rx.get(i), gv = sg[at];
                    const float d = p.softplus ? softplus(v) : v;
                    odx[i] = fmaf(d, s.x, skip[i] * gv);
                    float dd = fmaf(xv, s.x, s.y);
                    if (p.softplus) dd *= sigmoid(v);
                    odt[i] = dd;
                    aD[i] = fmaf(gv, xv, aD[i]);
                    ab[i] += dd;
                    if (z) {
                        const float zv = rz.get(i), s1 = sigmoid(zv);
                        oz[i] = rdy.get(i) * fmaf(skip[i], xv, sy[at]) * s1 * fmaf(zv, 1.f - s1, 1.f);
                    }
                }
                store_run(p.dx, t0 + lr, odx);
                store_run(p.ddt, t0 + lr, odt);
                if (z) store_run(p.dz, t0 + lr, oz);
            }
            for (int i = tid; i < kTile * 2 * N; i += kThreads) {
                const int t = t0 + i / (2 * N);
                float s = 0.f;
#pragma unroll
                for (int w = 0; w < S::kWarps; ++w) s += sred[w * kTile * 2 * N + i];
                if (t < tend) p.pBC[(((size_t)cb * p.B + stream) * p.T + t) * 2 * N + i % (2 * N)] = s;
            }
            __syncthreads();
        }
    }
    const size_t at = (size_t)stream * p.nseg + g;
    if constexpr (SUMMARY) {
        if (!live) return;
        store_state(p.eloc, at, e);
        if (q == 0) p.dsum[at * p.D + c] = dsum;
    } else {
        if (live) {
            store_state(p.pA, at, dA);
            if (g == 0 && p.dS0) store_state(p.dS0, stream, e);
        }
        // the 16 tokens' parts of dDskip and dbias of each channel, through shared memory
        float *sd = reinterpret_cast<float *>(sdx);
#pragma unroll
        for (int i = 0; i < E && lr < kTile; ++i) {
            sd[lr * kRow + lc + i] = aD[i];
            sg[lr * kRow + lc + i] = ab[i];
        }
        __syncthreads();
        for (int i = tid; i < 2 * CH; i += kThreads) {
            const int cc = i % CH;
            const float *src = i < CH ? sd : sg;
            float s = 0.f;
            for (int r = 0; r < kTile; ++r) s += src[r * kRow + cc];
            if (c0 + cc < p.D) p.pD[(at * 2 + i / CH) * p.D + c0 + cc] = s;
        }
    }
}

// dB and dC: the blocks' sums, in the order of the blocks. rows = B T; one thread per value.
template <typename T>
__global__ void ssm_reduce_bc_kernel(const float *pBC, long long rows, int N, int ncb, T *dBm, T *dCm)
{
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x, n = rows * 2 * N;
    if (i >= n) return;
    float s = 0.f;
    for (int b = 0; b < ncb; ++b) s += pBC[b * n + i];
    const long long row = i / (2 * N);
    const int j = (int)(i % (2 * N));
    if (j < N) store_one(dBm + row * N + j, s);
    else store_one(dCm + row * N + j - N, s);
}

// dA, dDskip and dbias: the sums over segments and batch entries, in their order.
__global__ void ssm_reduce_param_kernel(const float *pA, const float *pD, int parts, int D, int N, float *dA, float *dD,
                                        float *dbias)
{
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x, nA = (long long)D * N;
    if (i < nA) {
        float s = 0.f;
        for (int k = 0; k < parts; ++k) s += pA[k * nA + i];
        dA[i] = s;
    } else if (i < nA + 2LL * D) {
        const long long j = i - nA;  // dDskip, then dbias
        float *out = j < D ? dD : dbias;
        if (!out) return;
        float s = 0.f;
        for (int k = 0; k < parts; ++k) s += pD[k * 2LL * D + j];
        out[j < D ? j : j - D] = s;
    }
}

bool runs_aligned(const void *p, long long ld, int esz, int bytes)
{
    return !p || ((reinterpret_cast<uintptr_t>(p) % bytes) == 0 && (ld * esz) % bytes == 0);
}

template <typename T, int N>
cudaError_t launch_bwd(const SsmArgs &a, const SsmGrads &g, const BwdParams &p, cudaStream_t st)
{
    using S = BwdShape<N>;
    const int bytes = S::E * (int)sizeof(T) < 16 ? S::E * (int)sizeof(T) : 16;
    auto ok = [&](const void *q, long long ld) { return runs_aligned(q, ld, sizeof(T), bytes); };
    const bool vec = a.D % S::E == 0 && bytes >= 4 && ok(a.x, a.ldx) && ok(a.dt, a.lddt) && ok(a.z, a.ldz) &&
                     ok(g.dy, a.D) && ok(g.dx, a.D) && ok(g.ddt, a.D) && ok(g.dz, a.D);
    auto run = [&](auto *kern, int segments) -> cudaError_t {
        const int smem = S::kFloats * (int)sizeof(float);
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kern<<<dim3(p.ncb * a.B, segments), kThreads, smem, st>>>(p);
        return cudaGetLastError();
    };
    cudaError_t e = cudaSuccess;
    if (p.nseg > 1)
        e = vec ? run(ssm_backward_kernel<T, N, true, true>, p.nseg - 1)
                : run(ssm_backward_kernel<T, N, false, true>, p.nseg - 1);
    if (e != cudaSuccess) return e;
    e = vec ? run(ssm_backward_kernel<T, N, true, false>, p.nseg) : run(ssm_backward_kernel<T, N, false, false>, p.nseg);
    if (e != cudaSuccess) return e;
    const long long rows = (long long)a.B * a.T, nbc = rows * 2 * N;
    ssm_reduce_bc_kernel<T><<<(unsigned)((nbc + 255) / 256), 256, 0, st>>>(p.pBC, rows, N, p.ncb,
                                                                          static_cast<T *>(g.dBm),
                                                                          static_cast<T *>(g.dCm));
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long np = (long long)a.D * (N + 2);
    ssm_reduce_param_kernel<<<(unsigned)((np + 255) / 256), 256, 0, st>>>(p.pA, p.pD, a.B * p.nseg, a.D, N, g.dA, g.dD,
                                                                         g.dbias);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_bwd_n(const SsmArgs &a, const SsmGrads &g, const BwdParams &p, cudaStream_t st)
{
    switch (a.N) {
    case 8: return launch_bwd<T, 8>(a, g, p, st);
    case 16: return launch_bwd<T, 16>(a, g, p, st);
    case 32: return launch_bwd<T, 32>(a, g, p, st);
    default: return launch_bwd<T, 64>(a, g, p, st);
    }
}

// The backward's workspace, in this order; every part starts on 256 bytes.
struct Layout {
    size_t scan, saved, eloc, dsum, pBC, pA, pD, total;
};
Layout layout(int B, int T, int D, int N, bool have_saved)
{
    const SsmSplit s = ssm_split(B, T, D, N);
    const size_t ncb = (size_t)(D + 1024 / N - 1) / (1024 / N), parts = (size_t)B * s.nseg;
    const size_t nchunk = (size_t)(T + kSsmChunk - 1) / kSsmChunk;
    size_t at = 0;
    auto take = [&](size_t floats) { const size_t r = at; at += (floats * 4 + 255) / 256 * 256; return r; };
    Layout l;
    l.scan = take(have_saved ? 0 : ssm_scan_workspace_bytes(B, T, D, N) / 4);
    l.saved = take(have_saved ? 0 : B * nchunk * D * N);
    l.eloc = take(s.nseg > 1 ? parts * D * N : 0);
    l.dsum = take(s.nseg > 1 ? parts * D : 0);
    l.pBC = take(ncb * B * T * 2 * N);
    l.pA = take(parts * D * N);
    l.pD = take(parts * 2 * D);
    l.total = at;
    return l;
}

}  // namespace

size_t ssm_backward_workspace_bytes(int B, int T, int D, int N, bool have_saved_states)
{
    return layout(B, T, D, N, have_saved_states).total;
}

cudaError_t launch_ssm_backward(const SsmArgs &a, const SsmGrads &g, cudaStream_t st)
{
    const Layout l = layout(a.B, a.T, a.D, a.N, a.saved_states != nullptr);
    unsigned char *ws = static_cast<unsigned char *>(a.workspace);
    auto part = [&](size_t off) { return reinterpret_cast<float *>(ws + off); };
    const float *saved = a.saved_states;
    if (!saved) {
        SsmArgs f = a;
        f.y = nullptr;
        f.S_T = nullptr;
        f.z = nullptr;
        f.saved_states = part(l.saved);
        f.workspace = part(l.scan);
        const cudaError_t e = launch_ssm_scan(f, st);
        if (e != cudaSuccess) return e;
        saved = f.saved_states;
    }
    const SsmSplit s = ssm_split(a.B, a.T, a.D, a.N);
    BwdParams p;
    p.B = a.B; p.T = a.T; p.D = a.D; p.seg = s.seg; p.nseg = s.nseg;
    p.nchunk = (a.T + kSsmChunk - 1) / kSsmChunk;
    p.ncb = (a.D + 1024 / a.N - 1) / (1024 / a.N);
    p.softplus = a.softplus;
    p.x = a.x; p.dt = a.dt; p.z = a.z; p.Bm = a.Bm; p.Cm = a.Cm; p.dy = g.dy;
    p.ldx = a.ldx; p.lddt = a.lddt; p.ldz = a.ldz; p.ldb = a.ldb; p.ldc = a.ldc;
    p.A = a.A; p.Dskip = a.Dskip; p.bias = a.dt_bias; p.dS_T = g.dS_T; p.saved = saved;
    p.dx = g.dx; p.ddt = g.ddt; p.dz = g.dz; p.dS0 = g.dS0;
    p.eloc = part(l.eloc); p.dsum = part(l.dsum); p.pBC = part(l.pBC); p.pA = part(l.pA); p.pD = part(l.pD);
    return a.bf16 ? launch_bwd_n<__nv_bfloat16>(a, g, p, st) : launch_bwd_n<float>(a, g, p, st);
}

}  // namespace gdr2
