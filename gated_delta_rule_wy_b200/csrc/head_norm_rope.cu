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
// write backward). d / 8 lanes own a row of d channels; a lane holds both members of four pairs, so that the
// rotation needs no shuffles, and with the weight folded into the angles a pair costs four multiplications. The lanes
// take a few heads of one token at a time, whose sums are taken by one butterfly that halves the values with each
// step. What the lanes need next is copied to shared memory asynchronously, two tasks ahead, by the lane
// that uses it: with loads into registers the forward took 38 us and the backward 72 us for 4 x 4096 tokens of 16 + 2 heads
// of 128 channels in bf16, with the copies 27 us (5.6 TB/s) and 43 us (5.3 TB/s).

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr2_launch.h"
#include "seq_ops.h"

namespace gdr2 {
namespace {

using namespace seq;

constexpr int kThreads = 256;
constexpr int kMaxBlocks = 1024;  // of the backward: one partial weight gradient each, and one for the other side
constexpr int kStages = 3;  // tasks whose copies are under way, one of them at hand
// heads per task: what their registers allow at two blocks per SM. (bf16 runs two; in fp32 three stages of rows are 120 KB of
// shared memory a block, so that one runs at a time and a grid for two takes two rounds.)
constexpr int heads_per_task(bool backward) { return backward ? 2 : 4; }

struct Side {
    int H, chunks, blocks;  // heads, tasks per token, blocks
    const void *x, *dy;
    long long ld;
    const float *weight;
    void *out;
};

struct NormParams {
    int tokens, T, R, P, first;
    int norm;
    float eps;
    const float *cos_sin;
    const int *positions;
    Side side[2];
    float *part;  // backward: [blocks][d], queries' blocks first
    unsigned *status;
};

// A lane's eight channels as four pairs (a, b), two pairs per 64-bit register. Half-split: a and b are runs
// of four channels, R / 2 apart (past R: two neighbouring runs). Interleaved: eight consecutive channels.
// In shared memory they are pieces of at most 16 bytes, each kThreads pieces apart: a warp's lie side by side.
template <typename T, bool IL> struct Row8 {
    static constexpr int kBytes = IL || sizeof(T) == 4 ? 16 : 8;  // of a piece
    static constexpr int kPieces = 8 * sizeof(T) / kBytes;
    static constexpr int kSize = 8 * sizeof(T) * kThreads;        // of a row of all threads

    // this thread's pieces of `row` into `to` (its first piece's place)
    __device__ __forceinline__ static void fetch(unsigned char *to, const T *row, int ca, int cb)
    {
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
            copy_async<kBytes>(to + i * kThreads * kBytes, row + (kPieces == 1 || i == 0 ? ca : cb));
    }
    __device__ __forceinline__ static void get(const unsigned char *from, f32x2 (&a)[2], f32x2 (&b)[2])
    {
        float v[8];
        if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 w = *reinterpret_cast<const float4 *>(from + i * kThreads * kBytes);
                v[4 * i] = w.x; v[4 * i + 1] = w.y; v[4 * i + 2] = w.z; v[4 * i + 3] = w.w;
            }
        } else {
            Raw<T, 8> r;
            if constexpr (IL) {
                const uint4 w = *reinterpret_cast<const uint4 *>(from);
                r.w[0] = w.x; r.w[1] = w.y; r.w[2] = w.z; r.w[3] = w.w;
            } else {
                const uint2 lo = *reinterpret_cast<const uint2 *>(from);
                const uint2 hi = *reinterpret_cast<const uint2 *>(from + kThreads * kBytes);
                r.w[0] = lo.x; r.w[1] = lo.y; r.w[2] = hi.x; r.w[3] = hi.y;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = r.get(i);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            a[i] = IL ? pair(v[4 * i], v[4 * i + 2]) : pair(v[2 * i], v[2 * i + 1]);
            b[i] = IL ? pair(v[4 * i + 1], v[4 * i + 3]) : pair(v[4 + 2 * i], v[4 + 2 * i + 1]);
        }
    }
};
template <typename T, bool IL>
__device__ __forceinline__ void store_row8(T *row, int ca, int cb, const f32x2 (&a)[2], const f32x2 (&b)[2])
{
    float va[4], vb[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        split(a[i], va[2 * i], va[2 * i + 1]);
        split(b[i], vb[2 * i], vb[2 * i + 1]);
    }
    if constexpr (IL) {
        const float v[8] = {va[0], vb[0], va[1], vb[1], va[2], vb[2], va[3], vb[3]};
        store_vec<T, 8>(row + ca, v);
    } else {
        store_vec<T, 4>(row + ca, va);
        store_vec<T, 4>(row + cb, vb);
    }
}

// Sums of NV values over groups of LANES lanes, in every lane.
template <int LANES, int NV> __device__ __forceinline__ void row_sums(float (&v)[NV], int lane)
{
    constexpr unsigned all = 0xffffffffu;
    int m = LANES / 2;
#pragma unroll
    for (int w = NV / 2; w >= 1; w /= 2, m /= 2) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < w; ++i)
            v[i] = (up ? v[i + w] : v[i]) + __shfl_xor_sync(all, up ? v[i] : v[i + w], m);
    }
    float s = v[0];  // of value lane / (LANES / NV)
#pragma unroll
    for (int k = LANES / NV / 2; k >= 1; k /= 2) s += __shfl_xor_sync(all, s, k);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = __shfl_sync(all, s, (lane & ~(LANES - 1)) + i * (LANES / NV));
}

// shared memory: per stage the task's rows (x, backward dy too), its cosines and its sines
template <typename T, bool BACKWARD> constexpr int stage_bytes()
{
    return (heads_per_task(BACKWARD) * (BACKWARD ? 2 : 1) * 8 * (int)sizeof(T) + 32) * kThreads;
}

// A task: kHeads heads of one token. Its rows and angles are copied kStages - 1 tasks ahead by the lanes that use
// them, so that nothing but a lane's own copies is ever waited for; its position is read one task before that.
template <typename T, int D, bool BACKWARD, bool IL>
__global__ void __launch_bounds__(kThreads, 2) head_norm_kernel(const __grid_constant__ NormParams p)
{
    using Row = Row8<T, IL>;
    constexpr int LANES = D / 8, GROUPS = kThreads / LANES, PER_WARP = 32 / LANES, HB = heads_per_task(BACKWARD);
    extern __shared__ __align__(16) unsigned char smem[];
    const int lane = threadIdx.x & 31, l = lane % LANES, grp = threadIdx.x / LANES;
    const bool keys = (int)blockIdx.x >= p.side[0].blocks;
    const Side &sd = p.side[keys];
    const int block = blockIdx.x - (keys ? p.side[0].blocks : 0);
    const bool turns = 8 * l < p.R;  // the lane's pairs are among the first R channels
    const int ca = IL ? 8 * l : turns ? 4 * l : p.R + 8 * (l - p.R / 8), cb = IL || !turns ? ca + 4 : ca + p.R / 2;
    f32x2 wa[2], wb[2], acca[2], accb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int a0 = IL ? ca + 4 * i : ca + 2 * i, a1 = IL ? a0 + 2 : a0 + 1;
        const int b0 = IL ? a0 + 1 : cb + 2 * i, b1 = IL ? b0 + 2 : b0 + 1;
        wa[i] = sd.weight ? pair(__ldg(sd.weight + a0), __ldg(sd.weight + a1)) : pair(1.f, 1.f);
        wb[i] = sd.weight ? pair(__ldg(sd.weight + b0), __ldg(sd.weight + b1)) : pair(1.f, 1.f);
        acca[i] = accb[i] = 0;
    }
    const float scale = p.norm == 1 ? 1.f / D : 1.f;
    // This group's tasks are first, first + step, ...; a warp's groups run their loops together (shuffles need every
    // lane), and a group past the last task does that one again without storing.
    const int tasks = p.tokens * sd.chunks, step = sd.blocks * GROUPS, first = block * GROUPS + grp;
    const int rounds = (tasks - (first - grp % PER_WARP) + step - 1) / step;
    const int dtoken = step / sd.chunks, dchunk = step % sd.chunks;
    struct Task {
        int token, chunk;
    };
    auto advance = [&](Task &k) {
        k.token += dtoken;
        k.chunk += dchunk;
        if (k.chunk >= sd.chunks) { k.chunk -= sd.chunks; ++k.token; }
    };
    auto position = [&](const Task &k) {
        const int t = min(k.token, p.tokens - 1);
        return !turns ? 0 : p.positions ? __ldg(p.positions + t) : p.first + t % p.T;
    };
    unsigned char *const rows = smem + threadIdx.x * Row::kBytes;
    unsigned char *const angles = smem + kStages * HB * (BACKWARD ? 2 : 1) * Row::kSize + threadIdx.x * 16;
    auto row_at = [&](int stage, int i) { return rows + (stage * HB * (BACKWARD ? 2 : 1) + i) * Row::kSize; };
    auto angle_at = [&](int stage, int i) { return angles + (stage * 2 + i) * 16 * kThreads; };
    auto fetch = [&](const Task &k, int pos, int stage) {
        const int tok = min(k.token, p.tokens - 1);
        const T *x = static_cast<const T *>(sd.x) + tok * sd.ld;
        const T *dy = static_cast<const T *>(sd.dy) + (size_t)tok * sd.H * D;
#pragma unroll
        for (int i = 0; i < HB; ++i) {  // heads past the last read it again
            const int h = min(k.chunk * HB + i, sd.H - 1) * D;
            Row::fetch(row_at(stage, i), x + h, ca, cb);
            if constexpr (BACKWARD) Row::fetch(row_at(stage, HB + i), dy + h, ca, cb);
        }
        if (turns && pos >= 0 && pos < p.P) {
            const float *row = p.cos_sin + (size_t)pos * p.R + 4 * l;
            copy_async<16>(angle_at(stage, 0), row);
            copy_async<16>(angle_at(stage, 1), row + p.R / 2);
        }
        copies_commit();
    };
    Task head{first / sd.chunks, first % sd.chunks}, tail = head;  // the next task to copy, and to compute
    int pos[kStages], next = position(head);                       // of the tasks under way, and of `head`
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        pos[i] = next;
        fetch(head, pos[i], i);
        advance(head);
        next = position(head);
    }
    for (int round = 0; round < rounds; round += kStages)
#pragma unroll
        for (int stage = 0; stage < kStages; ++stage) {
            if (round + stage >= rounds) break;
            constexpr int kLast = kStages - 1;
            const int into = (stage + kLast) % kStages;
            pos[into] = next;
            fetch(head, pos[into], into);  // the stage that was computed last
            advance(head);
            next = position(head);
            copies_wait<kLast>();
            const bool ok = tail.token < p.tokens;
            const int tok = ok ? tail.token : 0, h0 = tail.chunk * HB, h1 = ok ? sd.H : 0;
            advance(tail);
            float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
            if (turns) {
                if (pos[stage] >= 0 && pos[stage] < p.P) {
                    c = *reinterpret_cast<const float4 *>(angle_at(stage, 0));
                    s = *reinterpret_cast<const float4 *>(angle_at(stage, 1));
                } else if (ok) {  // reported; the row keeps its norm and is not turned
                    atomicOr(p.status, kStatusBadPosition);
                }
            }
            const f32x2 cs[2] = {pair(c.x, c.y), pair(c.z, c.w)}, sn[2] = {pair(s.x, s.y), pair(s.z, s.w)};
            const f32x2 neg[2] = {pair(-s.x, -s.y), pair(-s.z, -s.w)};
            float sums[BACKWARD ? 2 * HB : HB];
            f32x2 a[HB][2], b[HB][2];
            [[maybe_unused]] f32x2 ga[BACKWARD ? HB : 1][2], gb[BACKWARD ? HB : 1][2];
#pragma unroll
            for (int k = 0; k < HB; ++k) {
                Row::get(row_at(stage, k), a[k], b[k]);
                float lo, hi;
                split(fma2(b[k][1], b[k][1], fma2(b[k][0], b[k][0], fma2(a[k][1], a[k][1], mul2(a[k][0], a[k][0])))), lo,
                      hi);
                sums[BACKWARD ? 2 * k : k] = lo + hi;
                if constexpr (BACKWARD) {
                    f32x2 ya[2], yb[2], dot = 0;
                    Row::get(row_at(stage, HB + k), ya, yb);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {  // turned back
                        ga[k][i] = fma2(yb[i], sn[i], mul2(ya[i], cs[i]));
                        gb[k][i] = fma2(ya[i], neg[i], mul2(yb[i], cs[i]));
                        const f32x2 da = mul2(ga[k][i], wa[i]);
                        dot = i ? fma2(da, a[k][i], dot) : mul2(da, a[k][i]);
                        dot = fma2(mul2(gb[k][i], wb[i]), b[k][i], dot);
                    }
                    split(dot, lo, hi);
                    sums[2 * k + 1] = lo + hi;
                }
            }
            if (p.norm) row_sums<LANES>(sums, lane);
            T *out = static_cast<T *>(sd.out) + (size_t)tok * sd.H * D;
            f32x2 aa[2], ab[2], ba[2], bb[2];  // y_a = a aa + b ab, y_b = a ba + b bb, but for the norm
            if constexpr (!BACKWARD) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    aa[i] = mul2(wa[i], cs[i]);
                    ab[i] = mul2(wb[i], neg[i]);
                    ba[i] = mul2(wa[i], sn[i]);
                    bb[i] = mul2(wb[i], cs[i]);
                }
            }
#pragma unroll
            for (int k = 0; k < HB; ++k) {
                const int h = h0 + k;
                const float inv = p.norm ? rsqrtf(fmaf(sums[BACKWARD ? 2 * k : k], scale, p.eps)) : 1.f;
                const f32x2 inv2 = pair(inv, inv);
                f32x2 oa[2], ob[2];
                if constexpr (!BACKWARD) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const f32x2 va = mul2(a[k][i], inv2), vb = mul2(b[k][i], inv2);
                        oa[i] = fma2(vb, ab[i], mul2(va, aa[i]));
                        ob[i] = fma2(va, ba[i], mul2(vb, bb[i]));
                    }
                } else {
                    const float f = p.norm ? -sums[2 * k + 1] * inv * scale : 0.f;
                    const f32x2 f2 = pair(f, f);
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const f32x2 va = mul2(a[k][i], inv2), vb = mul2(b[k][i], inv2);
                        if (h < h1) {  // a head read again may hold infinities, which zero would not clear
                            acca[i] = fma2(ga[k][i], va, acca[i]);
                            accb[i] = fma2(gb[k][i], vb, accb[i]);
                        }
                        oa[i] = mul2(inv2, fma2(va, f2, mul2(ga[k][i], wa[i])));
                        ob[i] = mul2(inv2, fma2(vb, f2, mul2(gb[k][i], wb[i])));
                    }
                }
                if (h < h1) store_row8<T, IL>(out + (size_t)h * D, ca, cb, oa, ob);
            }
        }
    copies_wait<0>();
    if constexpr (BACKWARD) {
        __syncthreads();
        float *sm = reinterpret_cast<float *>(smem);  // [GROUPS][D]
        store_row8<float, IL>(sm + grp * D, ca, cb, acca, accb);
        __syncthreads();
        for (int i = threadIdx.x; i < D; i += kThreads) {
            float s = 0.f;
            for (int k = 0; k < GROUPS; ++k) s += sm[k * D + i];
            p.part[(size_t)blockIdx.x * D + i] = s;
        }
    }
}

// dweight of both sides: one warp per value over its blocks' parts, always the same order.
__global__ void __launch_bounds__(256) head_norm_dweight_kernel(const float *part, int qblocks, int kblocks, int d,
                                                                float *dq, float *dk)
{
    const int lane = threadIdx.x & 31, i = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= 2 * d) return;
    const float *src = part + (i < d ? i : (size_t)qblocks * d + i - d);
    const int blocks = i < d ? qblocks : kblocks;
    float s = 0.f;
    for (int b = lane; b < blocks; b += 32) s += src[(size_t)b * d];
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
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
    constexpr int GROUPS = kThreads / (D / 8), HB = heads_per_task(BACKWARD);
    const int sms = sm_count();
    NormParams p;
    p.tokens = (int)a.tokens;
    p.T = a.T > 0 ? a.T : 1;
    p.R = a.R; p.P = a.P; p.first = a.first;
    p.norm = a.norm; p.eps = a.eps;
    p.cos_sin = a.cos_sin; p.positions = a.positions;
    p.status = a.status;
    p.part = static_cast<float *>(a.workspace);
    const long long chunks[2] = {(a.side[0].H + HB - 1) / HB, (a.side[1].H + HB - 1) / HB};  // tasks per token
    const long long cap = 2LL * sms < kMaxBlocks ? 2LL * sms : kMaxBlocks, all = chunks[0] + chunks[1];
    for (int s = 0; s < 2; ++s) {
        const HeadNormSide &h = a.side[s];
        const long long want = (a.tokens * chunks[s] + GROUPS - 1) / GROUPS;
        long long share = all ? (cap * chunks[s] + all / 2) / all : 0;  // of the resident blocks, as of the work
        if (share < 1) share = 1;
        p.side[s] = Side{h.H, (int)(chunks[s] ? chunks[s] : 1), (int)(want < share ? want : share), h.x, h.dy, h.ld, h.weight,
                         h.out};
    }
    const int blocks = p.side[0].blocks + p.side[1].blocks;
    if (blocks > 0) {
        constexpr int smem = kStages * stage_bytes<T, BACKWARD>();
        auto *kern = a.interleaved ? head_norm_kernel<T, D, BACKWARD, true> : head_norm_kernel<T, D, BACKWARD, false>;
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kern<<<blocks, kThreads, smem, st>>>(p);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (BACKWARD && (a.side[0].dweight || a.side[1].dweight)) {
        head_norm_dweight_kernel<<<(2 * D + 7) / 8, 256, 0, st>>>(p.part, p.side[0].blocks, p.side[1].blocks, D,
                                                                 a.side[0].dweight, a.side[1].dweight);
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

size_t head_norm_backward_workspace_bytes(int d) { return (size_t)(kMaxBlocks + 2) * d * sizeof(float); }
cudaError_t launch_head_norm_rope(const HeadNormArgs &a, cudaStream_t st) { return dispatch<false>(a, st); }
cudaError_t launch_head_norm_rope_backward(const HeadNormArgs &a, cudaStream_t st) { return dispatch<true>(a, st); }

}  // namespace gdr2
