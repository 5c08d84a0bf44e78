// ssm_scan.cu -- the selective state-space scan: a diagonal recurrence per channel c and
// state n whose step size, input and output vectors depend on the token,
//
//   D_t[c] = softplus(dt_t[c] + bias[c])              (or dt + bias)
//   h_t[c, n] = exp(D_t[c] A[c, n]) h_{t-1}[c, n] + D_t[c] B_t[n] x_t[c]
//   y_t[c] = (sum_n C_t[n] h_t[c, n] + Dskip[c] x_t[c]) * silu(z_t[c])
//
// over whole sequences (dense or packed), and one token at a time on resident states.
// All arithmetic is fp32.
//
// What bounds it: one exponential per (token, channel, state) -- 16 per 8 bytes of bf16
// tokens moved at N = 16 -- so the scan is bound by the special-function and FMA pipes, not by
// HBM; the single-token step reads and writes its state and is bound by HBM.
//
// Work split: N / 4 lanes per channel, four states in registers each (float4 loads of B and
// C from shared memory, four independent chains), 256 threads walking a segment of the time
// axis in tiles of 32 tokens. A tile's step sizes are formed once per (token, channel) by
// the threads that load them, and the same threads finish y from the scan's sums, so x and
// z stay in registers. Where the channels alone do not fill the GPU the time axis is cut in
// segments: a first launch gives each segment's final state from zero and the sum of its
// step sizes -- its transition is exp(A sum D), nothing else need be kept -- and the second
// starts every segment from the composition of the ones before it.

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
constexpr int kTile = 32;  // tokens per tile

struct ScanParams {
    int T, D, nseq;              // tokens per stream, channels, sequences
    int seg;                     // tokens per segment (a multiple of kTile)
    int nseg;                    // segments per stream
    int nchunk;                  // saved states per stream
    bool softplus;
    const int *cu;               // packed: sequence s is tokens cu[s] .. cu[s + 1] - 1
    const void *x, *dt, *z, *Bm, *Cm;
    long long ldx, lddt, ldz, ldb, ldc;  // elements from one token to the next
    const float *A, *Dskip, *bias, *S0;
    void *y;
    float *S_T, *saved;
    float *hloc;                 // [streams][nseg][D][N] final states of segments from zero
    float *dsum;                 // [streams][nseg][D] sums of their step sizes
};

template <typename T, int N> struct ScanShape {
    static constexpr int L = N / 4;            // lanes per channel
    static constexpr int CH = kThreads / L;    // channels per block
    static constexpr int E = CH / 8;           // consecutive channels a thread loads of one token
    static constexpr int kPad = 8;             // y's four tokens of a step fall in different banks
    static constexpr int kRow = CH + kPad;
};

// Sum over the L lanes of a channel of four tokens' partial sums; lanes 0 .. min(L, 4) - 1 end
// up with the totals they write (L = 2: two tokens per lane).
template <int L> __device__ __forceinline__ void reduce4(const float (&p)[4], int q, float (&out)[2], int &tok)
{
    const bool b0 = q & 1;
    float k0 = b0 ? p[2] : p[0], k1 = b0 ? p[3] : p[1];
    const float s0 = b0 ? p[0] : p[2], s1 = b0 ? p[1] : p[3];
    k0 += __shfl_xor_sync(0xffffffffu, s0, 1);
    k1 += __shfl_xor_sync(0xffffffffu, s1, 1);
    tok = b0 ? 2 : 0;
    if constexpr (L >= 4) {
        const bool b1 = q & 2;
        float k = b1 ? k1 : k0;
        const float s = b1 ? k0 : k1;
        k += __shfl_xor_sync(0xffffffffu, s, 2);
        if constexpr (L >= 8) k += __shfl_xor_sync(0xffffffffu, k, 4);
        if constexpr (L >= 16) k += __shfl_xor_sync(0xffffffffu, k, 8);
        tok += b1 ? 1 : 0;
        out[0] = k;
    } else {
        out[0] = k0;
        out[1] = k1;
    }
}

template <typename T, int N, bool VEC, bool SUMMARY>
__global__ void __launch_bounds__(kThreads) ssm_scan_kernel(ScanParams p)
{
    using S = ScanShape<T, N>;
    constexpr int L = S::L, CH = S::CH, E = S::E, kRow = S::kRow;
    constexpr int kBC = kTile * N / kThreads;  // elements of B (and of C) per thread
    __shared__ __align__(16) float2 sdx[kTile * kRow];  // (D, D x); then y in .x
    __shared__ __align__(16) float sB[kTile * N];
    __shared__ __align__(16) float sC[SUMMARY ? 4 : kTile * N];
    __shared__ unsigned smask[2];
    __shared__ int sseq[kTile];

    const int tid = threadIdx.x;
    const int ncb = (p.D + CH - 1) / CH;
    const int g = blockIdx.y, stream = blockIdx.x / ncb;
    const int c0 = (blockIdx.x % ncb) * CH;
    const int tbeg = g * p.seg, tend = min(p.T, tbeg + p.seg);
    // this thread's chain: channel c, states 4 q .. 4 q + 3
    const int ch = tid / L, q = tid % L, c = c0 + ch;
    const bool live = c < p.D;
    // and the run of a tile it loads and finishes: token lr, channels c0 + lc .. + E - 1
    const int lr = tid / 8, lc = (tid % 8) * E;
    const int lvalid = min(E, p.D - (c0 + lc));

    float A2[4] = {0.f, 0.f, 0.f, 0.f}, h[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
        const float4 a = *reinterpret_cast<const float4 *>(p.A + (size_t)c * N + 4 * q);
        A2[0] = a.x * kLog2e; A2[1] = a.y * kLog2e; A2[2] = a.z * kLog2e; A2[3] = a.w * kLog2e;
    }
    auto load_state = [&](const float *base, size_t index, float (&v)[4]) {
        const float4 a = *reinterpret_cast<const float4 *>(base + (index * p.D + c) * N + 4 * q);
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    };
    auto store_state = [&](float *base, size_t index) {
        *reinterpret_cast<float4 *>(base + (index * p.D + c) * N + 4 * q) = make_float4(h[0], h[1], h[2], h[3]);
    };
    auto initial = [&](int s) {  // the state before sequence s
        if (p.S0 && live) load_state(p.S0, s, h);
        else h[0] = h[1] = h[2] = h[3] = 0.f;
    };
    // the state entering this segment
    if (!p.cu && g == 0) initial(stream);
    if (!SUMMARY && g > 0 && live) {
        int first = 0;  // the segment that holds the first token of the sequence at hand
        if (p.cu) first = min(g, max(0, __ldg(p.cu + find_sequence(p.cu, p.nseq, tbeg))) / p.seg);
        if (first < g) {
            load_state(p.hloc, (size_t)stream * p.nseg + first, h);
            for (int i = first + 1; i < g; ++i) {
                const size_t at = (size_t)stream * p.nseg + i;
                const float ds = p.dsum[at * p.D + c];
                float o[4];
                load_state(p.hloc, at, o);
#pragma unroll
                for (int k = 0; k < 4; ++k) h[k] = fmaf(ex2(ds * A2[k]), h[k], o[k]);
            }
        }
    }
    float bias[E], skip[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = p.bias && i < lvalid ? __ldg(p.bias + c0 + lc + i) : 0.f;
        skip[i] = !SUMMARY && p.Dskip && i < lvalid ? __ldg(p.Dskip + c0 + lc + i) : 0.f;
    }

    const T *x = static_cast<const T *>(p.x), *dt = static_cast<const T *>(p.dt), *z = static_cast<const T *>(p.z);
    const T *Bm = static_cast<const T *>(p.Bm), *Cm = static_cast<const T *>(p.Cm);
    T *y = static_cast<T *>(p.y);
    auto load_run = [&](const T *base, long long ld, int t, Raw<T, E> &r) {
        if (t >= tend || lvalid <= 0) { r.zero(); return; }
        const T *src = base + ((size_t)stream * p.T + t) * ld + c0 + lc;
        if constexpr (VEC) r.load_vec(src);
        else r.load_each(src, lvalid);
    };
    Raw<T, E> rx, rdt, rz, nx, ndt, nz;
    float nb[kBC], nc[kBC];
    auto fetch = [&](int t0) {
        load_run(x, p.ldx, t0 + lr, nx);
        load_run(dt, p.lddt, t0 + lr, ndt);
        if constexpr (!SUMMARY)
            if (z) load_run(z, p.ldz, t0 + lr, nz);
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            const int r = (tid + i * kThreads) / N, n = (tid + i * kThreads) % N, t = t0 + r;
            const size_t row = (size_t)stream * p.T + t;
            nb[i] = t < tend ? load_one(Bm + row * p.ldb + n) : 0.f;
            if constexpr (!SUMMARY) nc[i] = t < tend ? load_one(Cm + row * p.ldc + n) : 0.f;
        }
    };
    float dsum = 0.f;
    fetch(tbeg);
    for (int t0 = tbeg; t0 < tend; t0 += kTile) {
        rx = nx; rdt = ndt; rz = nz;
        // step sizes of this thread's run; tokens past the segment and channels past D are inert (D = 0)
        const bool run_ok = t0 + lr < tend;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            const float v = rdt.get(i) + bias[i];
            const float d = run_ok && i < lvalid ? (p.softplus ? softplus(v) : v) : 0.f;
            sdx[lr * kRow + lc + i] = make_float2(d, d * rx.get(i));
        }
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            sB[tid + i * kThreads] = nb[i];
            if constexpr (!SUMMARY) sC[tid + i * kThreads] = nc[i];
        }
        if (p.cu && tid < 32) {
            const int t = t0 + tid;
            bool first = false, last = false;
            if (t < tend) {
                const int s = find_sequence(p.cu, p.nseq, t);
                sseq[tid] = s;
                first = __ldg(p.cu + s) == t;
                last = __ldg(p.cu + s + 1) == t + 1;
            }
            const unsigned mf = __ballot_sync(0xffffffffu, first), ml = __ballot_sync(0xffffffffu, last);
            if (tid == 0) { smask[0] = mf; smask[1] = ml; }
        }
        __syncthreads();
        if (t0 + kTile < tend) fetch(t0 + kTile);
        unsigned mf = 0, ml = 0;
        if (p.cu) { mf = smask[0]; ml = smask[1]; }
        const bool edges = (mf | ml) != 0;
#pragma unroll 2
        for (int tt = 0; tt < kTile; tt += 4) {
            if (!SUMMARY && p.saved && tt % kSsmChunk == 0 && t0 + tt < tend && live)
                store_state(p.saved, (size_t)stream * p.nchunk + (t0 + tt) / kSsmChunk);
            float part[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = tt + k;
                if (edges && ((mf >> t) & 1u)) initial(sseq[t]);
                const float2 dx = sdx[t * kRow + ch];
                const float4 b = *reinterpret_cast<const float4 *>(sB + t * N + 4 * q);
                h[0] = fmaf(ex2(dx.x * A2[0]), h[0], dx.y * b.x);
                h[1] = fmaf(ex2(dx.x * A2[1]), h[1], dx.y * b.y);
                h[2] = fmaf(ex2(dx.x * A2[2]), h[2], dx.y * b.z);
                h[3] = fmaf(ex2(dx.x * A2[3]), h[3], dx.y * b.w);
                if constexpr (SUMMARY) {
                    dsum += dx.x;
                } else {
                    const float4 cv = *reinterpret_cast<const float4 *>(sC + t * N + 4 * q);
                    part[k] = fmaf(cv.x, h[0], cv.y * h[1]) + fmaf(cv.z, h[2], cv.w * h[3]);
                    if (edges && ((ml >> t) & 1u) && p.S_T && live) store_state(p.S_T, sseq[t]);
                }
            }
            if constexpr (!SUMMARY) {
                float out[2];
                int tok;
                reduce4<L>(part, q, out, tok);  // every lane has read its step's (D, D x) before
                if (q < 4) {
                    sdx[(tt + tok) * kRow + ch].x = out[0];
                    if constexpr (L == 2) sdx[(tt + tok + 1) * kRow + ch].x = out[1];
                }
            }
        }
        __syncthreads();
        if constexpr (!SUMMARY) {
            if (run_ok && lvalid > 0 && y) {
                float o[E];
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    o[i] = fmaf(skip[i], rx.get(i), sdx[lr * kRow + lc + i].x);
                    if (z) { const float zv = rz.get(i); o[i] *= zv * sigmoid(zv); }
                }
                T *dst = y + ((size_t)stream * p.T + t0 + lr) * p.D + c0 + lc;
                if constexpr (VEC) store_vec<T, E>(dst, o);
                else store_each<T, E>(dst, o, lvalid);
            }
        }
    }
    if (!live) return;
    if constexpr (SUMMARY) {
        const size_t at = (size_t)stream * p.nseg + g;
        store_state(p.hloc, at);
        if (q == 0) p.dsum[at * p.D + c] = dsum;
    } else if (!p.cu && tend == p.T && p.S_T) {
        store_state(p.S_T, stream);
    }
}

// Packed sequences without tokens keep their state (or get zeros): one block per sequence.
__global__ void ssm_empty_kernel(const int *cu, const float *S0, float *S_T, size_t n)
{
    const int s = blockIdx.x;
    if (__ldg(cu + s) != __ldg(cu + s + 1)) return;
    for (size_t i = threadIdx.x; i < n; i += blockDim.x) S_T[s * n + i] = S0 ? S0[s * n + i] : 0.f;
}

// ---------------------------------------------------------------- one token
struct StepParams {
    int D;
    bool softplus;
    const void *x, *dt, *z, *Bm, *Cm;
    long long ldx, lddt, ldz, ldb, ldc;
    const float *A, *Dskip, *bias;
    float *S;
    void *y;
};

// N / 4 lanes per channel, four states each, kPer channels per thread in flight: the state
// is read and written once (128 bytes per channel at N = 16 against 8 of tokens).
template <typename T, int N, int kPer>
__global__ void __launch_bounds__(kThreads) ssm_step_kernel(StepParams p)
{
    constexpr int L = N / 4, CH = kThreads / L;
    const int tid = threadIdx.x, q = tid % L;
    const int seq = blockIdx.x;
    const int cb = blockIdx.y * CH * kPer + tid / L;
    float4 h[kPer], a[kPer];
    float xv[kPer], dv[kPer], zv[kPer];
    const T *x = static_cast<const T *>(p.x) + (size_t)seq * p.ldx;
    const T *dt = static_cast<const T *>(p.dt) + (size_t)seq * p.lddt;
    const T *z = p.z ? static_cast<const T *>(p.z) + (size_t)seq * p.ldz : nullptr;
    const T *Bm = static_cast<const T *>(p.Bm) + (size_t)seq * p.ldb + 4 * q;
    const T *Cm = static_cast<const T *>(p.Cm) + (size_t)seq * p.ldc + 4 * q;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int c = cb + k * CH;
        if (c < p.D) {
            h[k] = *reinterpret_cast<const float4 *>(p.S + ((size_t)seq * p.D + c) * N + 4 * q);
            a[k] = *reinterpret_cast<const float4 *>(p.A + (size_t)c * N + 4 * q);
            xv[k] = load_one(x + c);
            dv[k] = load_one(dt + c);
            zv[k] = z ? load_one(z + c) : 0.f;
        }
    }
    float b[4], cv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) { b[i] = load_one(Bm + i); cv[i] = load_one(Cm + i); }
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
        const int c = cb + k * CH;
        float s = 0.f, o = 0.f;
        if (c < p.D) {
            float d = dv[k] + (p.bias ? __ldg(p.bias + c) : 0.f);
            if (p.softplus) d = softplus(d);
            const float u = d * xv[k], d2 = d * kLog2e;
            h[k].x = fmaf(ex2(d2 * a[k].x), h[k].x, u * b[0]);
            h[k].y = fmaf(ex2(d2 * a[k].y), h[k].y, u * b[1]);
            h[k].z = fmaf(ex2(d2 * a[k].z), h[k].z, u * b[2]);
            h[k].w = fmaf(ex2(d2 * a[k].w), h[k].w, u * b[3]);
            *reinterpret_cast<float4 *>(p.S + ((size_t)seq * p.D + c) * N + 4 * q) = h[k];
            s = fmaf(cv[0], h[k].x, cv[1] * h[k].y) + fmaf(cv[2], h[k].z, cv[3] * h[k].w);
        }
#pragma unroll
        for (int m = 1; m < L; m <<= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
        if (c < p.D && q == 0) {
            o = fmaf(p.Dskip ? __ldg(p.Dskip + c) : 0.f, xv[k], s);
            if (z) o *= zv[k] * sigmoid(zv[k]);
            store_one(static_cast<T *>(p.y) + (size_t)seq * p.D + c, o);
        }
    }
}

// ---------------------------------------------------------------- host
int sm_count()
{
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

bool runs_aligned(const void *p, long long ld, int esz, int bytes)
{
    return !p || ((reinterpret_cast<uintptr_t>(p) % bytes) == 0 && (ld * esz) % bytes == 0);
}

template <typename T, int N>
cudaError_t launch_scan(const SsmArgs &a, const ScanParams &p, cudaStream_t st)
{
    using S = ScanShape<T, N>;
    const int streams = a.cu_seqlens ? 1 : a.B;
    const unsigned cb = (unsigned)((a.D + S::CH - 1) / S::CH);
    const int bytes = S::E * (int)sizeof(T) < 16 ? S::E * (int)sizeof(T) : 16;
    const bool vec = a.D % S::E == 0 && runs_aligned(a.x, a.ldx, sizeof(T), bytes) &&
                     runs_aligned(a.dt, a.lddt, sizeof(T), bytes) && runs_aligned(a.z, a.ldz, sizeof(T), bytes) &&
                     runs_aligned(a.y, a.D, sizeof(T), bytes);
    if (p.nseg > 1) {
        const dim3 grid(cb * streams, p.nseg - 1);
        if (vec) ssm_scan_kernel<T, N, true, true><<<grid, kThreads, 0, st>>>(p);
        else ssm_scan_kernel<T, N, false, true><<<grid, kThreads, 0, st>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    const dim3 grid(cb * streams, p.nseg);
    if (vec) ssm_scan_kernel<T, N, true, false><<<grid, kThreads, 0, st>>>(p);
    else ssm_scan_kernel<T, N, false, false><<<grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_scan_n(const SsmArgs &a, const ScanParams &p, cudaStream_t st)
{
    switch (a.N) {
    case 8: return launch_scan<T, 8>(a, p, st);
    case 16: return launch_scan<T, 16>(a, p, st);
    case 32: return launch_scan<T, 32>(a, p, st);
    default: return launch_scan<T, 64>(a, p, st);
    }
}

template <typename T>
cudaError_t launch_step_n(const SsmArgs &a, const StepParams &p, cudaStream_t st)
{
    constexpr int kPer = 4;
    const unsigned per = (unsigned)(kThreads / (a.N / 4) * kPer);
    const dim3 grid(a.B, (a.D + per - 1) / per);
    switch (a.N) {
    case 8: ssm_step_kernel<T, 8, kPer><<<grid, kThreads, 0, st>>>(p); break;
    case 16: ssm_step_kernel<T, 16, kPer><<<grid, kThreads, 0, st>>>(p); break;
    case 32: ssm_step_kernel<T, 32, kPer><<<grid, kThreads, 0, st>>>(p); break;
    default: ssm_step_kernel<T, 64, kPer><<<grid, kThreads, 0, st>>>(p); break;
    }
    return cudaGetLastError();
}

}  // namespace

// Segments of the time axis: enough blocks to fill the GPU four times over, segments of at
// least 64 tokens, and none where the channels alone give two blocks per SM.
SsmSplit ssm_split(int streams, int T, int D, int N)
{
    const long long blocks = (long long)streams * ((D + 1024 / N - 1) / (1024 / N));
    const int sms = sm_count();
    long long g = blocks >= 2LL * sms ? 1 : (4LL * sms + blocks - 1) / (blocks > 0 ? blocks : 1);
    const long long most = (T + 63) / 64;
    if (g > most) g = most;
    if (g < 1) g = 1;
    SsmSplit s;
    s.seg = (int)(((T + g - 1) / g + kTile - 1) / kTile * kTile);
    if (s.seg < kTile) s.seg = kTile;
    s.nseg = (T + s.seg - 1) / s.seg;
    if (s.nseg < 1) s.nseg = 1;
    return s;
}

size_t ssm_scan_workspace_bytes(int streams, int T, int D, int N)
{
    const SsmSplit s = ssm_split(streams, T, D, N);
    if (s.nseg <= 1) return 0;
    const size_t n = (size_t)streams * s.nseg * D;
    return (n * (N + 1) * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_ssm_scan(const SsmArgs &a, cudaStream_t st)
{
    const int streams = a.cu_seqlens ? 1 : a.B;
    if (a.T > 0 && streams > 0 && a.D > 0) {
        const SsmSplit s = ssm_split(streams, a.T, a.D, a.N);
        ScanParams p;
        p.T = a.T; p.D = a.D; p.nseq = a.B;
        p.seg = s.seg; p.nseg = s.nseg;
        p.nchunk = (a.T + kSsmChunk - 1) / kSsmChunk;
        p.softplus = a.softplus;
        p.cu = a.cu_seqlens;
        p.x = a.x; p.dt = a.dt; p.z = a.z; p.Bm = a.Bm; p.Cm = a.Cm;
        p.ldx = a.ldx; p.lddt = a.lddt; p.ldz = a.ldz; p.ldb = a.ldb; p.ldc = a.ldc;
        p.A = a.A; p.Dskip = a.Dskip; p.bias = a.dt_bias; p.S0 = a.S0;
        p.y = a.y; p.S_T = a.S_T; p.saved = a.saved_states;
        p.hloc = static_cast<float *>(a.workspace);
        p.dsum = p.hloc + (size_t)streams * s.nseg * a.D * a.N;
        const cudaError_t e = a.bf16 ? launch_scan_n<__nv_bfloat16>(a, p, st) : launch_scan_n<float>(a, p, st);
        if (e != cudaSuccess) return e;
    }
    if (a.cu_seqlens && a.S_T && a.B > 0 && a.D > 0) {
        ssm_empty_kernel<<<a.B, 256, 0, st>>>(a.cu_seqlens, a.S0, a.S_T, (size_t)a.D * a.N);
        return cudaGetLastError();
    }
    return cudaSuccess;
}

cudaError_t launch_ssm_step(const SsmArgs &a, cudaStream_t st)
{
    StepParams p;
    p.D = a.D;
    p.softplus = a.softplus;
    p.x = a.x; p.dt = a.dt; p.z = a.z; p.Bm = a.Bm; p.Cm = a.Cm;
    p.ldx = a.ldx; p.lddt = a.lddt; p.ldz = a.ldz; p.ldb = a.ldb; p.ldc = a.ldc;
    p.A = a.A; p.Dskip = a.Dskip; p.bias = a.dt_bias;
    p.S = a.S_T;
    p.y = a.y;
    return a.bf16 ? launch_step_n<__nv_bfloat16>(a, p, st) : launch_step_n<float>(a, p, st);
}

}  // namespace gdr2
