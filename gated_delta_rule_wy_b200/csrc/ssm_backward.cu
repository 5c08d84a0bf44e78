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
// Work split as in the forward: a block owns 32 channels over a segment of the time axis, in tiles
// of kSsmChunk tokens from the last to the first. Scanning warps (lane = channel, four states each) form a
// tile's states again from the one saved before it, eight tokens at a time in registers (the first eight
// twice: 32 registers instead of 64 let two blocks share an SM), and walk back; helper warps form the step sizes
// and gates of the tile to the left and the token gradients of the tile to the right meanwhile.
//
// What bounds it: the latency of the scanning warps (eight per SM, an instruction every 4 to 5 cycles of each; shared
// memory's data path 74% busy, the special-function unit 37%). 2 x 4096 tokens of 2048 channels, N = 16, bf16: 575 us, of 737
// with the forward. Measured against it: 16 tokens' states in registers and one block per SM 1057 us in all, two channels
// per lane 880, B and C read at one address 744, blocks of 64 channels 716 to 810.
//
// The sums over channels (dB, dC) are taken over a warp's 32 lanes by shuffles that halve the values with each step.
// Lane l holds its four states in the order j ^ (l & 3): in the first two steps every lane then keeps its low
// half and gives its high half, without selects (shared memory has B and C in the four orders). The blocks' sums
// are added by a last kernel in a fixed order: no atomics, the same bits each time.
//
// Segments of the time axis as in the forward, from the right: the first launch walks the last segment
// whole and gives the others' own part of the gradient that leaves them to the left and the sums of their
// step sizes; the second starts each of the others from the composition of those to its right.

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "gdr2_launch.h"
#include "seq_ops.h"

namespace gdr2 {
namespace {

using namespace seq;

constexpr int kCh = 32;         // channels per block: the lanes of a warp
constexpr int kTile = kSsmChunk;
constexpr int kHalf = kTile / 2;  // tokens whose states are in registers at a time
constexpr int kHelpers = 128;
constexpr int E = kTile * kCh / kHelpers;  // consecutive channels a helper has of one token
static_assert(E == 4, "a helper has four channels");

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
    static constexpr int G = N < 32 ? N / 4 : 8;    // scanning warps
    static constexpr int R = N / (4 * G);           // sets of four states a warp walks one after the other
    static constexpr int kBlock = 32 * G + kHelpers;
    static constexpr int kBlocks = N <= 16 ? 2 : 1; // per SM
    static constexpr int kDuRow = 2 * kCh + 8, kGRow = kCh + 4, kPRow = kCh * G + 4;
    static constexpr int kBCRow = 8 * N;            // of one token: B and C, of every four states the four orders
    // shared memory, in floats: (D, D x); g; B and C; the warps' parts of du, dD and y; the sums over channels;
    // what a helper keeps of its elements from their conversion to their gradients
    static constexpr int kDu = 0, kG = kDu + 2 * kTile * kDuRow, kBC = kG + 2 * kTile * kGRow;
    static constexpr int kPart = kBC + 2 * kTile * kBCRow, kSum = kPart + 2 * 3 * kTile * kPRow;
    static constexpr int kKeep = kSum + 2 * kTile * 2 * N;
    static constexpr int kFloats = kKeep + 3 * 5 * 4 * kHelpers;
    static constexpr int kRuns = N < 16 ? 1 : N / 16;  // runs of four elements of B and C per helper
};

// v[j] <-> v[j ^ order]: from the natural order of four states to a lane's and back
__device__ __forceinline__ void reorder(float (&v)[4], int order)
{
    const bool hi = order & 2, lo = order & 1;
    const float a = hi ? v[2] : v[0], b = hi ? v[3] : v[1], c = hi ? v[0] : v[2], d = hi ? v[1] : v[3];
    v[0] = lo ? b : a; v[1] = lo ? a : b; v[2] = lo ? d : c; v[3] = lo ? c : d;
}

// Sums over the 32 lanes of b and c, four states in the lane's order: lane l, and every 8th from it,
// returns the sum of state l & 3, of b where l & 4 is 0 and of c where not.
__device__ __forceinline__ float channel_sum(const float (&b)[4], const float (&c)[4], int lane)
{
    constexpr unsigned all = 0xffffffffu;
    const float b0 = b[0] + __shfl_xor_sync(all, b[2], 2), b1 = b[1] + __shfl_xor_sync(all, b[3], 2);
    const float c0 = c[0] + __shfl_xor_sync(all, c[2], 2), c1 = c[1] + __shfl_xor_sync(all, c[3], 2);
    const float bs = b0 + __shfl_xor_sync(all, b1, 1), cs = c0 + __shfl_xor_sync(all, c1, 1);
    const bool up = lane & 4;
    float v = (up ? cs : bs) + __shfl_xor_sync(all, up ? bs : cs, 4);
    v += __shfl_xor_sync(all, v, 8);
    return v + __shfl_xor_sync(all, v, 16);
}

// SUMMARY: the segment's own part of the gradient that leaves it to the left, and sum D.
template <typename T, int N, bool VEC, bool SUMMARY>
__device__ __forceinline__ void walk_segment(const BwdParams &p, int g, float *smem)
{
    using S = BwdShape<N>;
    constexpr int G = S::G, R = S::R;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int stream = blockIdx.x / p.ncb, cb = blockIdx.x % p.ncb, c0 = cb * kCh;
    const int tbeg = g * p.seg, tend = min(p.T, tbeg + p.seg);
    const int nt = (tend - tbeg + kTile - 1) / kTile;
    const size_t row0 = (size_t)stream * p.T, part_at = (size_t)stream * p.nseg + g;

    if (warp < G) {  // ---------------------------------------------------------------- scan
        const int c = c0 + lane, order = lane & 3;
        const bool live = c < p.D;
        float A2[R][4] = {};
        f32x2 e[R][2], A[R][2], dA[R][2];
        auto load_state = [&](const float *base, size_t index, int r, f32x2 (&v)[2]) {
            const float4 a = *reinterpret_cast<const float4 *>(base + (index * p.D + c) * N + 4 * (warp * R + r));
            float w[4] = {a.x, a.y, a.z, a.w};
            reorder(w, order);
            v[0] = pair(w[0], w[1]);
            v[1] = pair(w[2], w[3]);
        };
        auto store_state = [&](float *base, size_t index, int r, const f32x2 (&v)[2]) {
            float w[4];
            split(v[0], w[0], w[1]);
            split(v[1], w[2], w[3]);
            reorder(w, order);
            *reinterpret_cast<float4 *>(base + (index * p.D + c) * N + 4 * (warp * R + r)) =
                make_float4(w[0], w[1], w[2], w[3]);
        };
        auto decay = [&](float d, int r, int k) { return pair(decay2(d, A2[r][2 * k]), decay2(d, A2[r][2 * k + 1])); };
#pragma unroll
        for (int r = 0; r < R; ++r) {
            e[r][0] = e[r][1] = A[r][0] = A[r][1] = dA[r][0] = dA[r][1] = 0;
            if (live) load_state(p.A, 0, r, A[r]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                float lo, hi;
                split(A[r][k], lo, hi);
                A[r][k] = pair(held(lo), held(hi));
                A2[r][2 * k] = decay_rate(lo);
                A2[r][2 * k + 1] = decay_rate(hi);
            }
            // e = a_{t+1} dh_{t+1}, the gradient that enters this segment from the right
            if (!live) continue;
            if (g == p.nseg - 1) {
                if (p.dS_T) load_state(p.dS_T, stream, r, e[r]);
            } else if (!SUMMARY) {
                load_state(p.eloc, (size_t)stream * p.nseg + p.nseg - 1, r, e[r]);
#pragma unroll 2
                for (int i = p.nseg - 2; i > g; --i) {
                    const size_t at = (size_t)stream * p.nseg + i;
                    const float ds = p.dsum[at * p.D + c];
                    f32x2 o[2];
                    load_state(p.eloc, at, r, o);
#pragma unroll
                    for (int k = 0; k < 2; ++k) e[r][k] = carry2(ds, A2[r][2 * k], A2[r][2 * k + 1], e[r][k], o[k]);
                }
            }
        }
        const float *sdu = smem + S::kDu + 4 * (lane / 2 ^ lane / 16) + 2 * (lane & 1), *sg = smem + S::kG + lane;
        const float *sbc = smem + S::kBC + 16 * warp * R + 4 * order;
        float *spart = smem + S::kPart + kCh * warp + lane;
        // its sum over the channels of one state of B or C; lanes with the same store the same
        float *ssum = smem + S::kSum + (lane & 4) / 4 * N + 4 * warp * R + order;
        float dsum = 0.f;
        f32x2 saved[R][2];  // the state before the next tile
        auto fetch_saved = [&](int it) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                saved[r][0] = saved[r][1] = 0;
                if (!SUMMARY && live && it >= 0)
                    load_state(p.saved, (size_t)stream * p.nchunk + tbeg / kTile + it, r, saved[r]);
            }
        };
        fetch_saved(nt - 1);
        for (int it = nt - 1; it >= 0; --it) {
            __syncthreads();
            const int buf = it & 1;
            auto du_at = [&](int t) { return *reinterpret_cast<const float2 *>(sdu + (buf * kTile + t) * S::kDuRow); };
            auto g_at = [&](int t) { return sg[(buf * kTile + t) * S::kGRow]; };
            auto bc_at = [&](int t, int which, int r, f32x2 (&v)[2]) {
                lds_pairs(sbc + (buf * kTile + t) * S::kBCRow + which * 4 * N + 16 * r, v[0], v[1]);
            };
            if constexpr (SUMMARY) {
#pragma unroll
                for (int t = kTile - 1; t >= 0; --t) {
                    const float d = du_at(t).x, gv = g_at(t);
                    const f32x2 gg = pair(gv, gv);
                    dsum += d;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        f32x2 cc[2];
                        bc_at(t, 1, r, cc);
#pragma unroll
                        for (int k = 0; k < 2; ++k) e[r][k] = mul2(decay(d, r, k), fma2(cc[k], gg, e[r][k]));
                    }
                }
            } else {
                f32x2 first[R][2];
#pragma unroll
                for (int r = 0; r < R; ++r) { first[r][0] = saved[r][0]; first[r][1] = saved[r][1]; }
                fetch_saved(it - 1);
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    f32x2 sA[2] = {0, 0};  // the tile's part of dA: sums of sums round less than one long one
                    // the compiler reads shared memory anew behind this: it would keep every token's decays for
                    // the walk back instead of forming them again, in 64 registers
                    auto forget = [] { asm volatile("" ::: "memory"); };
                    auto forward = [&](int t, const f32x2 (&from)[2], f32x2 (&to)[2]) {
                        const float2 du = du_at(t);
                        const f32x2 uu = pair(du.y, du.y);
                        f32x2 bb[2];
                        bc_at(t, 0, r, bb);
#pragma unroll
                        for (int k = 0; k < 2; ++k) to[k] = fma2(decay(du.x, r, k), from[k], mul2(uu, bb[k]));
                    };
                    struct Token {
                        float2 du;
                        float g;
                        f32x2 b[2], c[2];
                    };
                    auto load = [&](int t, Token &k) {
                        k.du = du_at(t);
                        k.g = g_at(t);
                        bc_at(t, 0, r, k.b);
                        bc_at(t, 1, r, k.c);
                    };
                    // the tokens from kFrom on, with the state before them
                    auto walk = [&](auto from, const f32x2 (&before)[2]) {
                        constexpr int kFrom = decltype(from)::value;
                        f32x2 h[kHalf][2];
                        forward(kFrom, before, h[0]);
#pragma unroll
                        for (int i = 1; i < kHalf; ++i) forward(kFrom + i, h[i - 1], h[i]);
                        forget();
                        Token now, next;
                        load(kFrom + kHalf - 1, now);
#pragma unroll
                        for (int i = kHalf - 1; i >= 0; --i) {
                            const int t = kFrom + i;
                            if (i > 0) load(t - 1, next);
                            const f32x2 dd = pair(now.du.x, now.du.x), uu = pair(now.du.y, now.du.y);
                            const f32x2 gg = pair(now.g, now.g);
                            f32x2 sdx = 0, sdd = 0, sy = 0;
                            float vb[4], vc[4];
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const f32x2 prev = i ? h[i ? i - 1 : 0][k] : before[k];
                                const f32x2 dh = fma2(now.c[k], gg, e[r][k]);
                                split(mul2(uu, dh), vb[2 * k], vb[2 * k + 1]);
                                split(mul2(gg, h[i][k]), vc[2 * k], vc[2 * k + 1]);
                                e[r][k] = mul2(decay(now.du.x, r, k), dh);
                                const f32x2 m = mul2(e[r][k], prev);
                                sA[k] = fma2(dd, m, sA[k]);
                                sdx = k ? fma2(now.b[k], dh, sdx) : mul2(now.b[k], dh);
                                sdd = k ? fma2(A[r][k], m, sdd) : mul2(A[r][k], m);
                                sy = k ? fma2(now.c[k], h[i][k], sy) : mul2(now.c[k], h[i][k]);
                            }
                            float *out = spart + (buf * 3 * kTile + t) * S::kPRow;
                            auto put = [&](int which, f32x2 v) {
                                float lo, hi;
                                split(v, lo, hi);
                                float *o = out + which * kTile * S::kPRow;
                                *o = r ? *o + (lo + hi) : lo + hi;
                            };
                            put(0, sdx);
                            put(1, sdd);
                            put(2, sy);
                            ssum[(buf * kTile + t) * 2 * N + 4 * r] = channel_sum(vb, vc, lane);
                            now = next;
                        }
                    };
                    f32x2 middle[2] = {first[r][0], first[r][1]};
#pragma unroll
                    for (int t = 0; t < kHalf; ++t) forward(t, middle, middle);
                    forget();
                    walk(std::integral_constant<int, kHalf>{}, middle);
                    walk(std::integral_constant<int, 0>{}, first[r]);
#pragma unroll
                    for (int k = 0; k < 2; ++k) dA[r][k] = add2(dA[r][k], sA[k]);
                }
            }
        }
        if constexpr (!SUMMARY) __syncthreads();
        if (live) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (SUMMARY || (g == p.nseg - 1 && p.nseg > 1)) store_state(p.eloc, part_at, r, e[r]);
                if constexpr (!SUMMARY) {
                    store_state(p.pA, part_at, r, dA[r]);
                    if (g == 0 && p.dS0) store_state(p.dS0, stream, r, e[r]);
                }
            }
            if (SUMMARY && warp == 0) p.dsum[part_at * p.D + c] = dsum;
        }
        if constexpr (!SUMMARY) __syncthreads();
        return;
    }
    // ---------------------------------------------------------------- helpers
    const int hid = tid - 32 * G;
    const int lr = hid / (kCh / E), lc = hid % (kCh / E) * E;  // its token of a tile, its first channel
    const int lvalid = min(E, p.D - (c0 + lc));
    float bias[E], skip[E], aD[E], ab[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = p.bias && i < lvalid ? __ldg(p.bias + c0 + lc + i) : 0.f;
        skip[i] = p.Dskip && i < lvalid ? __ldg(p.Dskip + c0 + lc + i) : 0.f;
        aD[i] = ab[i] = 0.f;
    }
    const T *x = static_cast<const T *>(p.x), *dt = static_cast<const T *>(p.dt), *z = static_cast<const T *>(p.z);
    const T *dy = static_cast<const T *>(p.dy);
    // as in the forward, loads are never conditional: tokens past the segment and channels past D read the
    // last one, and are made inert when converted
    auto load_run = [&](const T *base, long long ld, int t, Raw<T, E> &r) {
        const T *row = base + (row0 + min(t, tend - 1)) * ld;
        if constexpr (VEC) r.load_vec(row + min(c0 + lc, p.D - E));
        else r.load_clamped(row, c0 + lc, p.D - 1);
    };
    struct Tokens {
        Raw<T, E> x, dt, z, dy;
        uint32_t bc[S::kRuns][4];
    };
    constexpr int kUnits = N / 2;  // runs of B and C of one token
    const int bu = hid % kUnits, br = hid / kUnits;
    constexpr int kRows = kHelpers / kUnits;
    const bool is_c = bu >= N / 4;
    const T *const bc_base = (is_c ? static_cast<const T *>(p.Cm) : static_cast<const T *>(p.Bm)) + bu % (N / 4) * 4;
    const long long bc_ld = is_c ? p.ldc : p.ldb;
    auto fetch = [&](int t0, Tokens &k) {
        load_run(dt, p.lddt, t0 + lr, k.dt);
        load_run(dy, p.D, t0 + lr, k.dy);
        load_run(x, p.ldx, t0 + lr, k.x);
        if (z) load_run(z, p.ldz, t0 + lr, k.z);
#pragma unroll
        for (int i = 0; i < S::kRuns; ++i) {
            const T *b = bc_base + (row0 + min(t0 + br + i * kRows, tend - 1)) * bc_ld;
#pragma unroll
            for (int j = 0; j < 4; ++j) k.bc[i][j] = load_bits(b + j);
        }
    };
    auto keep_at = [&](int it, int what) {  // four floats of this thread, of one tile
        return reinterpret_cast<float4 *>(smem + S::kKeep) + ((it % 3) * 5 + what) * kHelpers + hid;
    };
    auto convert = [&](const Tokens &tok, int it) {
        const int t0 = tbeg + it * kTile, buf = it & 1;
        const bool in = t0 + lr < tend;
        float d[E], sg[E], xv[E], gv[E], zf[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            d[i] = tok.dt.get(i) + bias[i];
            xv[i] = tok.x.get(i);
            gv[i] = tok.dy.get(i);
            sg[i] = 1.f;
            zf[i] = 0.f;
        }
        if (p.softplus)
#pragma unroll
            for (int i = 0; i < E; ++i) { sg[i] = softplus_slope(d[i]); d[i] = softplus(d[i]); }
        if (z)
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float zv = tok.z.get(i), s = sigmoid(zv);
                zf[i] = gv[i] * s * fmaf(zv, 1.f - s, 1.f);
                gv[i] *= zv * s;
            }
        float u[E];
#pragma unroll
        for (int i = 0; i < E; ++i) u[i] = d[i] * xv[i];
        if (t0 + kTile > tend || lvalid < E)
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (!in || i >= lvalid) d[i] = u[i] = gv[i] = 0.f;
        const int swap = lc / (kCh / 2);
        float4 *dst = reinterpret_cast<float4 *>(smem + S::kDu + (buf * kTile + lr) * S::kDuRow + 2 * lc);
        dst[swap] = make_float4(d[0], u[0], d[1], u[1]);
        dst[1 - swap] = make_float4(d[2], u[2], d[3], u[3]);
        auto four = [](const float (&v)[E]) { return make_float4(v[0], v[1], v[2], v[3]); };
        *reinterpret_cast<float4 *>(smem + S::kG + (buf * kTile + lr) * S::kGRow + lc) = four(gv);
        if constexpr (!SUMMARY) {
            *keep_at(it, 0) = four(d);
            *keep_at(it, 1) = four(gv);
            *keep_at(it, 2) = four(xv);
            *keep_at(it, 3) = four(sg);
            *keep_at(it, 4) = four(zf);
        }
#pragma unroll
        for (int i = 0; i < S::kRuns; ++i) {
            const int r = br + i * kRows;
            if (r >= kTile) continue;
            const bool m = t0 + r < tend;
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = m ? bits_value<T>(tok.bc[i][j]) : 0.f;
            // order j holds v[k ^ j]; neighbours write different j at a time, and so different banks
            float4 *o = reinterpret_cast<float4 *>(smem + S::kBC + (buf * kTile + r) * S::kBCRow) + 4 * bu;
            const int sw = bu / 2 & 3;
            reorder(v, sw);
            o[sw] = make_float4(v[0], v[1], v[2], v[3]);
            o[sw ^ 1] = make_float4(v[1], v[0], v[3], v[2]);
            o[sw ^ 2] = make_float4(v[2], v[3], v[0], v[1]);
            o[sw ^ 3] = make_float4(v[3], v[2], v[1], v[0]);
        }
    };
    auto finish = [&](int it) {
#pragma unroll
        for (int i = hid; i < kTile * N / 2; i += kHelpers) {  // the tile's sums over channels
            const int r = i / (N / 2), t = tbeg + it * kTile + r;
            const float4 v = *reinterpret_cast<const float4 *>(smem + S::kSum + (it & 1) * kTile * 2 * N + 4 * i);
            if (t < tend)
                *reinterpret_cast<float4 *>(p.pBC + ((size_t)cb * p.B * p.T + row0 + t) * 2 * N + i % (N / 2) * 4) = v;
        }
        const int t = tbeg + it * kTile + lr;
        if (t >= tend || lvalid <= 0) return;
        float s[3][E];
#pragma unroll
        for (int w = 0; w < 3; ++w) {
            const float *src = smem + S::kPart + (((it & 1) * 3 + w) * kTile + lr) * S::kPRow + lc;
#pragma unroll
            for (int i = 0; i < E; ++i) s[w][i] = 0.f;
#pragma unroll
            for (int k = 0; k < G; ++k) {
                const float4 v = *reinterpret_cast<const float4 *>(src + k * kCh);
                s[w][0] += v.x; s[w][1] += v.y; s[w][2] += v.z; s[w][3] += v.w;
            }
        }
        float d[E], gv[E], xv[E], sg[E], zf[E];
        auto get = [&](int what, float (&v)[E]) {
            const float4 a = *keep_at(it, what);
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        };
        get(0, d); get(1, gv); get(2, xv); get(3, sg); get(4, zf);
        float odx[E], odt[E], oz[E];
#pragma unroll
        for (int i = 0; i < E; ++i) {
            odx[i] = fmaf(d[i], s[0][i], skip[i] * gv[i]);
            odt[i] = fmaf(xv[i], s[0][i], s[1][i]) * sg[i];
            oz[i] = zf[i] * fmaf(skip[i], xv[i], s[2][i]);
            if (i < lvalid) {
                aD[i] = fmaf(gv[i], xv[i], aD[i]);
                ab[i] += odt[i];
            }
        }
        auto store_run = [&](void *base, const float (&v)[E]) {
            T *dst = static_cast<T *>(base) + (row0 + t) * p.D + c0 + lc;
            if constexpr (VEC) store_vec<T, E>(dst, v);
            else store_each<T, E>(dst, v, lvalid);
        };
        store_run(p.dx, odx);
        store_run(p.ddt, odt);
        if (z) store_run(p.dz, oz);
    };
    // the eight helpers of a token ask for the rows of the six inputs, kAhead tiles before their loads
    constexpr int kAhead = 3;
    const T *prow = x + c0;
    long long prl = p.ldx;
    switch (hid % 8) {
    case 1: prow = dt + c0; prl = p.lddt; break;
    case 2: if (z) { prow = z + c0; prl = p.ldz; } break;
    case 3: prow = dy + c0; prl = p.D; break;
    case 4: prow = static_cast<const T *>(p.Bm); prl = p.ldb; break;
    case 5: prow = static_cast<const T *>(p.Cm); prl = p.ldc; break;
    }
    auto prefetch = [&](int t0) {
        asm volatile("prefetch.global.L2 [%0];" ::"l"(prow + (row0 + max(t0 + lr, tbeg)) * prl));
    };
    Tokens tok;
    if (nt > 0) {
#pragma unroll
        for (int k = 1; k <= kAhead && k < nt; ++k) prefetch(tbeg + (nt - 1 - k) * kTile);
        fetch(tbeg + (nt - 1) * kTile, tok);
        convert(tok, nt - 1);
        if (nt > 1) fetch(tbeg + (nt - 2) * kTile, tok);
    }
    for (int it = nt - 1; it >= 0; --it) {
        __syncthreads();
        if (it > 0) convert(tok, it - 1);
        if (!SUMMARY && it < nt - 1) finish(it + 1);
        if (it > 1) fetch(tbeg + (it - 2) * kTile, tok);
        if (it > 1 + kAhead) prefetch(tbeg + (it - 2 - kAhead) * kTile);
    }
    if constexpr (!SUMMARY) {
        __syncthreads();
        if (nt > 0) finish(0);
        // the tokens' parts of dDskip and dbias of each channel, through shared memory
        float4 *sd = reinterpret_cast<float4 *>(smem + S::kBC), *sb = sd + kHelpers;
        sd[hid] = make_float4(aD[0], aD[1], aD[2], aD[3]);
        sb[hid] = make_float4(ab[0], ab[1], ab[2], ab[3]);
        __syncthreads();
        if (hid < 2 * kCh) {
            const float *src = reinterpret_cast<const float *>(hid < kCh ? sd : sb) + hid % kCh;
            float s = 0.f;
#pragma unroll
            for (int r = 0; r < kTile; ++r) s += src[r * kCh];
            const int c = c0 + hid % kCh;
            if (c < p.D) p.pD[(part_at * 2 + hid / kCh) * p.D + c] = s;
        }
    }
}

// FIRST (two segments or more): the last segment whole and the others' summaries, from the second on;
// otherwise all segments (one), or those up to the last but one.
template <typename T, int N, bool VEC, bool FIRST>
__global__ void __launch_bounds__(BwdShape<N>::kBlock, BwdShape<N>::kBlocks) ssm_backward_kernel(BwdParams p)
{
    extern __shared__ __align__(16) float smem[];
    if constexpr (FIRST) {
        if (blockIdx.y == 0) walk_segment<T, N, VEC, false>(p, p.nseg - 1, smem);
        else walk_segment<T, N, VEC, true>(p, blockIdx.y, smem);
    } else {
        walk_segment<T, N, VEC, false>(p, blockIdx.y, smem);
    }
}

struct ReduceParams {
    const float *pBC, *pA, *pD;
    long long rows;             // B T
    int N, D, ncb, parts;       // parts: segments and batch entries
    unsigned bc_blocks;         // the first blocks: dB and dC
    float *dA, *dD, *dbias;
};

// One thread per value, always in the same order: dB and dC over the blocks' channels, then dA, dDskip and dbias
// over segments and batch entries.
template <typename T> __global__ void __launch_bounds__(256) ssm_reduce_kernel(ReduceParams p, T *dBm, T *dCm)
{
    if (blockIdx.x < p.bc_blocks) {
        const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x, n = p.rows * 2 * p.N;
        if (i >= n) return;
        float s = 0.f;
#pragma unroll 8
        for (int b = 0; b < p.ncb; ++b) s += p.pBC[b * n + i];
        const long long row = i / (2 * p.N);
        const int j = (int)(i % (2 * p.N));
        if (j < p.N) store_one(dBm + row * p.N + j, s);
        else store_one(dCm + row * p.N + j - p.N, s);
        return;
    }
    const long long i = (long long)(blockIdx.x - p.bc_blocks) * blockDim.x + threadIdx.x, nA = (long long)p.D * p.N;
    if (i < nA) {
        float s = 0.f;
        for (int k = 0; k < p.parts; ++k) s += p.pA[k * nA + i];
        p.dA[i] = s;
    } else if (i < nA + 2LL * p.D) {
        const long long j = i - nA;  // dDskip, then dbias
        float *out = j < p.D ? p.dD : p.dbias;
        if (!out) return;
        float s = 0.f;
        for (int k = 0; k < p.parts; ++k) s += p.pD[k * 2LL * p.D + j];
        out[j < p.D ? j : j - p.D] = s;
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
    auto ok = [&](const void *q, long long ld) { return runs_aligned(q, ld, sizeof(T), E * (int)sizeof(T)); };
    const bool vec = a.D % E == 0 && ok(a.x, a.ldx) && ok(a.dt, a.lddt) && ok(a.z, a.ldz) && ok(g.dy, a.D) &&
                     ok(g.dx, a.D) && ok(g.ddt, a.D) && ok(g.dz, a.D);
    auto run = [&](auto *kern, int segments) -> cudaError_t {
        const int smem = S::kFloats * (int)sizeof(float);
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kern<<<dim3(p.ncb * a.B, segments), S::kBlock, smem, st>>>(p);
        return cudaGetLastError();
    };
    cudaError_t e = cudaSuccess;
    if (p.nseg > 1)
        e = vec ? run(ssm_backward_kernel<T, N, true, true>, p.nseg - 1)
                : run(ssm_backward_kernel<T, N, false, true>, p.nseg - 1);
    if (e != cudaSuccess) return e;
    const int rest = p.nseg > 1 ? p.nseg - 1 : 1;
    e = vec ? run(ssm_backward_kernel<T, N, true, false>, rest) : run(ssm_backward_kernel<T, N, false, false>, rest);
    if (e != cudaSuccess) return e;
    ReduceParams r;
    r.pBC = p.pBC; r.pA = p.pA; r.pD = p.pD;
    r.rows = (long long)a.B * a.T;
    r.N = N; r.D = a.D; r.ncb = p.ncb; r.parts = a.B * p.nseg;
    r.bc_blocks = (unsigned)((r.rows * 2 * N + 255) / 256);
    r.dA = g.dA; r.dD = g.dD; r.dbias = g.dbias;
    const unsigned more = (unsigned)(((long long)a.D * (N + 2) + 255) / 256);
    ssm_reduce_kernel<T><<<r.bc_blocks + more, 256, 0, st>>>(r, static_cast<T *>(g.dBm), static_cast<T *>(g.dCm));
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

int sm_count()
{
    int dev = 0, n = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    return n > 0 ? n : 148;
}

// Segments of the time axis, as in the forward. Of two launches the first runs a whole segment and g - 2 summaries
// per 32 channels, the second g - 1 whole ones; a summary costs kSummary of a whole token. The constants are those of
// N = 16, two blocks per SM; the other N take the same rule, which was not measured for them.
SsmSplit ssm_backward_split(int streams, int T, int D)
{
    constexpr double kAlone = 1.27, kSummary = 0.45;
    const long long blocks = (long long)streams * ((D + kCh - 1) / kCh);
    const int sms = sm_count(), tiles = (T + kTile - 1) / kTile;
    auto load = [&](long long n) {  // of n equal blocks, in tokens of one of two blocks that share an SM
        const long long k = (n + sms - 1) / sms;
        return k % 2 ? k - 1 + kAlone : (double)k;
    };
    auto cost = [&](int g) {
        const double tokens = (tiles + g - 1) / g * (double)kTile + 32.;
        if (g == 1) return tokens * load(blocks);
        const double f = (1. + kSummary * (g - 2)) / (g - 1);  // a first launch's block, on average
        return tokens * load(blocks * (g - 1)) * (1. + (f < kSummary ? kSummary : f)) + 2. * g;
    };
    int best = 1;
    for (int g = 2; g <= tiles && g <= 256; ++g)
        if (cost(g) < cost(best)) best = g;
    SsmSplit s;
    s.seg = (tiles + best - 1) / best * kTile;
    if (s.seg < kTile) s.seg = kTile;
    s.nseg = (T + s.seg - 1) / s.seg;
    if (s.nseg < 1) s.nseg = 1;
    return s;
}

// The backward's workspace, in this order; every part starts on 256 bytes.
struct Layout {
    size_t scan, saved, eloc, dsum, pBC, pA, pD, total;
};
Layout layout(int B, int T, int D, int N, bool have_saved)
{
    const SsmSplit s = ssm_backward_split(B, T, D);
    const size_t ncb = (size_t)(D + kCh - 1) / kCh, parts = (size_t)B * s.nseg;
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
    const SsmSplit s = ssm_backward_split(a.B, a.T, a.D);
    BwdParams p;
    p.B = a.B; p.T = a.T; p.D = a.D; p.seg = s.seg; p.nseg = s.nseg;
    p.nchunk = (a.T + kSsmChunk - 1) / kSsmChunk;
    p.ncb = (a.D + kCh - 1) / kCh;
    p.softplus = a.softplus;
    p.x = a.x; p.dt = a.dt; p.z = a.z; p.Bm = a.Bm; p.Cm = a.Cm; p.dy = g.dy;
    p.ldx = a.ldx; p.lddt = a.lddt; p.ldz = a.ldz; p.ldb = a.ldb; p.ldc = a.ldc;
    p.A = a.A; p.Dskip = a.Dskip; p.bias = a.dt_bias; p.dS_T = g.dS_T; p.saved = saved;
    p.dx = g.dx; p.ddt = g.ddt; p.dz = g.dz; p.dS0 = g.dS0;
    p.eloc = part(l.eloc); p.dsum = part(l.dsum); p.pBC = part(l.pBC); p.pA = part(l.pA); p.pD = part(l.pD);
    return a.bf16 ? launch_bwd_n<__nv_bfloat16>(a, g, p, st) : launch_bwd_n<float>(a, g, p, st);
}

}  // namespace gdr2
