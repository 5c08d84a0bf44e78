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
// What bounds it: one exponential per (token, channel, state) on the special-function unit, 16 per
// SM and cycle, and four for a (token, channel) (softplus and the gate): at N = 16 a floor of 172 us for 4 x 4096
// tokens of 2048 channels, against 41 us of HBM traffic. The single-token step reads and
// writes its state (18.7 us for 256 x 2048 x 16 states, 3.8 TB/s, 58% of the HBM rate): 58 warps per SM
// issue in 64% of the cycles, much of it for B and C, read element by element, and wait for loads 58% of their time.
//
// Work split: a block owns 32 channels over a segment of the time axis, in tiles of 32 tokens. N / 4
// scanning warps hold four states of each channel in registers, lane = channel: B and C are
// broadcast reads of shared memory, no shuffles, and a token costs a warp 4 exponentials and about 17
// other instructions. Four helper warps do what is done once per (token, channel): step sizes
// ahead of the scan, and behind it the sum of the warps' parts, the skip and the gate. (Lanes of one
// channel side by side, each token's work in the same threads, took 587 us; this form 254 us with
// two blocks per SM, 68% of the floor; helpers alone 127 us, scanning warps alone 162 us.)
//
// Where the channels do not fill the GPU the time axis is cut in g segments: a first launch scans the
// first segment whole and gives the others' final states from zero and the sums of their
// step sizes -- a segment's transition is exp(A sum D), nothing else need be kept -- and the second
// starts every later segment from the composition of the ones before it.

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

constexpr int kThreads = 256;   // of the single-token step
constexpr int kCh = 32;         // channels per block: the lanes of a warp
constexpr int kHelpers = 128;   // threads that convert tokens and finish outputs
constexpr int kTile = 32;       // tokens per tile
constexpr int E = kTile * kCh / kHelpers;  // consecutive channels a helper has of one token
static_assert(kTile % kSsmChunk == 0 && E == 8, "a tile is whole chunks");

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

template <int N> struct ScanShape {
    static constexpr int G = N / 4;                      // scanning warps
    static constexpr int kBlock = 32 * G + kHelpers;
    static constexpr int kStep = N == 64 ? 2 : 4;        // tokens whose shared-memory loads are in flight together
    static constexpr int kBlocks = N <= 16 ? 2 : 1;      // per SM
    // floats per token of (D, D x). The upper half's 16-byte chunks are swapped in pairs and rows are 8 floats
    // apart from a multiple of 32: chunks written together fall in different banks
    static constexpr int kDuRow = 2 * kCh + 8;
    static constexpr int kYRow = kCh * G + 4;            // of the warps' parts of y
    static constexpr int kDu = 0, kB = 2 * kTile * kDuRow, kC = kB + 2 * kTile * N, kY = kC + 2 * kTile * N;
    static constexpr int kFloats = kY + 2 * kTile * kYRow;
    static constexpr int kBC = N < 16 ? 1 : N / 16;      // runs of four elements of B (and C) per helper
};

// One block: 32 channels over one segment of one stream. The first N / 4 warps scan tile i, lane = channel,
// four states each; meanwhile the helpers turn tile i + 1 into (D, D x), finish the output of tile i - 1 and
// have the loads of tile i + 2 in flight. One barrier per tile.
template <typename T, int N, bool VEC, bool SUMMARY>
__device__ __forceinline__ void scan_segment(const ScanParams &p, int g, float *smem, unsigned (&smask)[2][2],
                                             int (&sseq)[2][kTile])
{
    using S = ScanShape<N>;
    constexpr int G = S::G, kBC = S::kBC, kStep = S::kStep;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int ncb = (p.D + kCh - 1) / kCh;
    const int stream = blockIdx.x / ncb, c0 = blockIdx.x % ncb * kCh;
    const int tbeg = g * p.seg, tend = min(p.T, tbeg + p.seg);
    const int nt = (tend - tbeg + kTile - 1) / kTile;

    if (!SUMMARY && p.cu && g == 0 && p.S_T)  // packed sequences without tokens keep their state, or get zeros
        for (int s = warp; s < p.nseq; s += S::kBlock / 32) {
            if (__ldg(p.cu + s) != __ldg(p.cu + s + 1)) continue;
            for (int i = lane; i < kCh * N / 4; i += 32) {
                const int c = c0 + i / (N / 4);
                const size_t at = ((size_t)s * p.D + c) * N + i % (N / 4) * 4;
                if (c < p.D)
                    *reinterpret_cast<float4 *>(p.S_T + at) =
                        p.S0 ? *reinterpret_cast<const float4 *>(p.S0 + at) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }

    if (warp < G) {  // ---------------------------------------------------------------- scan
        const int c = c0 + lane, q = warp;
        const bool live = c < p.D;
        float A2[4] = {0.f, 0.f, 0.f, 0.f};
        f32x2 h[2] = {0, 0};
        if (live) {
            const float4 a = *reinterpret_cast<const float4 *>(p.A + (size_t)c * N + 4 * q);
            A2[0] = decay_rate(a.x); A2[1] = decay_rate(a.y); A2[2] = decay_rate(a.z); A2[3] = decay_rate(a.w);
        }
        auto load_state = [&](const float *base, size_t index, f32x2 (&v)[2]) {
            const float4 a = *reinterpret_cast<const float4 *>(base + (index * p.D + c) * N + 4 * q);
            v[0] = pair(a.x, a.y);
            v[1] = pair(a.z, a.w);
        };
        auto store_state = [&](float *base, size_t index) {
            float4 a;
            split(h[0], a.x, a.y);
            split(h[1], a.z, a.w);
            *reinterpret_cast<float4 *>(base + (index * p.D + c) * N + 4 * q) = a;
        };
        auto decay = [&](float d, int k) { return pair(decay2(d, A2[2 * k]), decay2(d, A2[2 * k + 1])); };
        auto initial = [&](int s) {  // the state before sequence s
            if (p.S0 && live) load_state(p.S0, s, h);
            else h[0] = h[1] = 0;
        };
        // the state entering this segment
        if (!p.cu && g == 0) initial(stream);
        if (!SUMMARY && g > 0 && live) {
            int first = 0;  // the segment that holds the first token of the sequence at hand
            if (p.cu) first = min(g, max(0, __ldg(p.cu + find_sequence(p.cu, p.nseq, tbeg))) / p.seg);
            if (first < g) {
                load_state(p.hloc, (size_t)stream * p.nseg + first, h);
#pragma unroll 4
                for (int i = first + 1; i < g; ++i) {
                    const size_t at = (size_t)stream * p.nseg + i;
                    const float ds = p.dsum[at * p.D + c];
                    f32x2 o[2];
                    load_state(p.hloc, at, o);
#pragma unroll
                    for (int k = 0; k < 2; ++k) h[k] = carry2(ds, A2[2 * k], A2[2 * k + 1], h[k], o[k]);
                }
            }
        }
        struct Token {
            float2 du;
            f32x2 b[2], c[2];
        };
        const int chunk = lane / 2 ^ lane / 16;  // of this channel's (D, D x)
        const float *sdu = smem + S::kDu + 4 * chunk + 2 * (lane & 1), *sB = smem + S::kB + 4 * q, *sC = smem + S::kC + 4 * q;
        float *sy = smem + S::kY + kCh * q + lane;
        float dsum = 0.f;
        for (int it = 0; it < nt; ++it) {
            __syncthreads();
            const int buf = it & 1, t0 = tbeg + it * kTile;
            auto load = [&](int t, Token &k) {
                k.du = *reinterpret_cast<const float2 *>(sdu + (buf * kTile + t) * S::kDuRow);
                lds_pairs(sB + (buf * kTile + t) * N, k.b[0], k.b[1]);
                if constexpr (!SUMMARY) lds_pairs(sC + (buf * kTile + t) * N, k.c[0], k.c[1]);
            };
            unsigned mf = 0, ml = 0;
            if (p.cu) { mf = smask[buf][0]; ml = smask[buf][1]; }
            auto steps = [&](auto edges) {
                constexpr bool EDGES = decltype(edges)::value;
                Token now[kStep], next[kStep];
#pragma unroll
                for (int k = 0; k < kStep; ++k) load(k, now[k]);
#pragma unroll
                for (int st = 0; st < kTile; st += kStep) {
                    if (st + kStep < kTile)
#pragma unroll
                        for (int k = 0; k < kStep; ++k) load(st + kStep + k, next[k]);
                    if (!SUMMARY && st % kSsmChunk == 0 && p.saved && live && t0 + st < tend)
                        store_state(p.saved, (size_t)stream * p.nchunk + (t0 + st) / kSsmChunk);
#pragma unroll
                    for (int k = 0; k < kStep; ++k) {
                        const int t = st + k;
                        if constexpr (EDGES)
                            if ((mf >> t) & 1u) initial(sseq[buf][t]);
                        const float d = now[k].du.x;
                        const f32x2 u = pair(now[k].du.y, now[k].du.y);
                        h[0] = fma2(decay(d, 0), h[0], mul2(u, now[k].b[0]));
                        h[1] = fma2(decay(d, 1), h[1], mul2(u, now[k].b[1]));
                        if constexpr (SUMMARY) {
                            dsum += d;
                        } else {
                            float lo, hi;
                            split(fma2(now[k].c[0], h[0], mul2(now[k].c[1], h[1])), lo, hi);
                            sy[(buf * kTile + t) * S::kYRow] = lo + hi;
                            if constexpr (EDGES)
                                if (((ml >> t) & 1u) && p.S_T && live) store_state(p.S_T, sseq[buf][t]);
                        }
                    }
#pragma unroll
                    for (int k = 0; k < kStep; ++k) now[k] = next[k];
                }
            };
            if ((mf | ml) != 0) steps(std::true_type{});
            else steps(std::false_type{});
        }
        if constexpr (!SUMMARY) __syncthreads();
        if (!live) return;
        if (SUMMARY || (g == 0 && p.nseg > 2)) store_state(p.hloc, (size_t)stream * p.nseg + g);
        if (SUMMARY && q == 0) p.dsum[((size_t)stream * p.nseg + g) * p.D + c] = dsum;
        if (!SUMMARY && !p.cu && tend == p.T && p.S_T) store_state(p.S_T, stream);
        return;
    }
    // ---------------------------------------------------------------- helpers
    const int hid = tid - 32 * G;
    const int lr = hid / (kCh / E), lc = hid % (kCh / E) * E;  // its token of a tile, its first channel
    const int lvalid = min(E, p.D - (c0 + lc));
    float bias[E], skip[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        bias[i] = p.bias && i < lvalid ? __ldg(p.bias + c0 + lc + i) : 0.f;
        skip[i] = !SUMMARY && p.Dskip && i < lvalid ? __ldg(p.Dskip + c0 + lc + i) : 0.f;
    }
    const T *x = static_cast<const T *>(p.x), *dt = static_cast<const T *>(p.dt), *z = static_cast<const T *>(p.z);
    const T *Bm = static_cast<const T *>(p.Bm), *Cm = static_cast<const T *>(p.Cm);
    T *y = static_cast<T *>(p.y);
    // Loads are never conditional (a test before each would make them wait for one another): tokens past
    // the segment and channels past D read the last one, and are made inert when converted.
    const size_t row0 = (size_t)stream * p.T;
    auto load_run = [&](const T *base, long long ld, int t, Raw<T, E> &r) {
        const T *row = base + (row0 + min(t, tend - 1)) * ld;
        if constexpr (VEC) r.load_vec(row + min(c0 + lc, p.D - E));
        else r.load_clamped(row, c0 + lc, p.D - 1);
    };
    struct Tokens {
        Raw<T, E> x, dt;
        uint32_t b[kBC][4], c[kBC][4];
    };
    constexpr int kRows = kHelpers / (N / 4);  // rows of B that the helpers read at once, four elements each
    const int br = hid / (N / 4), bn = hid % (N / 4) * 4;
    auto four = [](const uint32_t (&v)[4], bool in) {
        return make_float4(in ? bits_value<T>(v[0]) : 0.f, in ? bits_value<T>(v[1]) : 0.f,
                           in ? bits_value<T>(v[2]) : 0.f, in ? bits_value<T>(v[3]) : 0.f);
    };
    auto fetch = [&](int t0, Tokens &k) {
        load_run(x, p.ldx, t0 + lr, k.x);
        load_run(dt, p.lddt, t0 + lr, k.dt);
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            const size_t row = row0 + min(t0 + br + i * kRows, tend - 1);
            const T *b = Bm + row * p.ldb + bn, *c = Cm + row * p.ldc + bn;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                k.b[i][j] = load_bits(b + j);
                if constexpr (!SUMMARY) k.c[i][j] = load_bits(c + j);
            }
        }
    };
    int seq_begin = 0x7fffffff, seq_end = 0;
    // the fetched tile into buffer `buf`; tokens past the segment and channels past D are inert
    // (D = 0: the decay is 1 and nothing is added)
    auto convert = [&](const Tokens &tok, int t0, int buf) {
        float4 *dst = reinterpret_cast<float4 *>(smem + S::kDu + (buf * kTile + lr) * S::kDuRow + 2 * lc);
        const int swap = lc / (kCh / 2);
        const bool in = t0 + lr < tend;
        float d[E];
#pragma unroll
        for (int i = 0; i < E; ++i) d[i] = tok.dt.get(i) + bias[i];
        if (p.softplus)
#pragma unroll
            for (int i = 0; i < E; ++i) d[i] = softplus(d[i]);
        float u[E];
#pragma unroll
        for (int i = 0; i < E; ++i) u[i] = d[i] * tok.x.get(i);
        if (t0 + kTile > tend || lvalid < E)
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (!in || i >= lvalid) d[i] = u[i] = 0.f;
#pragma unroll
        for (int i = 0; i < E; i += 2)
            dst[i / 2 + (i % 4 == 0 ? swap : -swap)] = make_float4(d[i], u[i], d[i + 1], u[i + 1]);
#pragma unroll
        for (int i = 0; i < kBC; ++i) {
            const int r = br + i * kRows, at = (buf * kTile + r) * N + bn;
            if (r < kTile) {
                *reinterpret_cast<float4 *>(smem + S::kB + at) = four(tok.b[i], t0 + r < tend);
                if constexpr (!SUMMARY) *reinterpret_cast<float4 *>(smem + S::kC + at) = four(tok.c[i], t0 + r < tend);
            }
        }
        if (p.cu && hid < 32) {  // packed: which of the tile's tokens begin and end a sequence
            const int t = t0 + hid;
            bool first = false, last = false;
            if (!(seq_begin < t0 && t0 + kTile < seq_end)) {  // not all of the tile inside the sequence last seen
                const int s = find_sequence(p.cu, p.nseq, min(t, tend - 1));
                sseq[buf][hid] = s;
                seq_begin = __ldg(p.cu + s);
                seq_end = __ldg(p.cu + s + 1);
                first = t < tend && seq_begin == t;
                last = t < tend && seq_end == t + 1;
                seq_begin = __shfl_sync(0xffffffffu, seq_begin, 31);  // of the tile's last token
                seq_end = __shfl_sync(0xffffffffu, seq_end, 31);
            }
            const unsigned mf = __ballot_sync(0xffffffffu, first), ml = __ballot_sync(0xffffffffu, last);
            if (hid == 0) { smask[buf][0] = mf; smask[buf][1] = ml; }
        }
    };
    struct Outer {
        Raw<T, E> x, z;
    };
    auto fetch_outer = [&](int t0, Outer &k) {
        if (SUMMARY || !y) return;
        load_run(x, p.ldx, t0 + lr, k.x);
        if (z) load_run(z, p.ldz, t0 + lr, k.z);
    };
    auto finish = [&](const Outer &k, int t0, int buf) {
        if (t0 + lr >= tend || lvalid <= 0 || !y) return;
        float o[E];
#pragma unroll
        for (int i = 0; i < E; ++i) o[i] = skip[i] * k.x.get(i);
        const float *src = smem + S::kY + (buf * kTile + lr) * S::kYRow + lc;
#pragma unroll
        for (int w = 0; w < G; ++w)
#pragma unroll
            for (int i = 0; i < E; i += 4) {
                const float4 v = *reinterpret_cast<const float4 *>(src + w * kCh + i);
                o[i] += v.x; o[i + 1] += v.y; o[i + 2] += v.z; o[i + 3] += v.w;
            }
        if (z)
#pragma unroll
            for (int i = 0; i < E; ++i) { const float zv = k.z.get(i); o[i] *= zv * sigmoid(zv); }
        T *dst = y + ((size_t)stream * p.T + t0 + lr) * p.D + c0 + lc;
        if constexpr (VEC) store_vec<T, E>(dst, o);
        else store_each<T, E>(dst, o, lvalid);
    };
    // Each of the four helpers of a token asks for one tensor's row, kAhead tiles before it is loaded: loads
    // then come from L2 and return before the next tile (from HBM they take longer than a tile's work).
    constexpr int kAhead = 3;
    const T *const pbase[4] = {x + c0, dt + c0, z ? z + c0 : x + c0, SUMMARY || hid % 8 < 4 ? Bm : Cm};
    const long long pld[4] = {p.ldx, p.lddt, z ? p.ldz : p.ldx, SUMMARY || hid % 8 < 4 ? p.ldb : p.ldc};
    const T *prow = pbase[0];
    long long prl = pld[0];
#pragma unroll
    for (int i = 1; i < 4; ++i)
        if (hid % 4 == i) { prow = pbase[i]; prl = pld[i]; }
    auto prefetch = [&](int t0) {
        const T *row = prow + (row0 + min(t0 + lr, tend - 1)) * prl;
        asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
    };
    Tokens tok;
    Outer out;
    if (nt > 0) {
#pragma unroll
        for (int k = 1; k <= kAhead; ++k) prefetch(tbeg + k * kTile);
        fetch(tbeg, tok);
        convert(tok, tbeg, 0);
        fetch(tbeg + kTile, tok);
    }
    for (int it = 0; it < nt; ++it) {
        __syncthreads();
        const int t0 = tbeg + it * kTile;
        convert(tok, t0 + kTile, (it + 1) & 1);
        if (!SUMMARY && it > 0) finish(out, t0 - kTile, (it - 1) & 1);
        fetch(t0 + 2 * kTile, tok);
        fetch_outer(t0, out);
        prefetch(t0 + (2 + kAhead) * kTile);
    }
    if constexpr (!SUMMARY) {
        __syncthreads();
        if (nt > 0) finish(out, tbeg + (nt - 1) * kTile, (nt - 1) & 1);
    }
}

// FIRST (three segments or more): the first segment whole and the others' summaries, up to the last
// but one; otherwise all segments (one), or those from the second on.
template <typename T, int N, bool VEC, bool FIRST>
__global__ void __launch_bounds__(ScanShape<N>::kBlock, ScanShape<N>::kBlocks) ssm_scan_kernel(ScanParams p)
{
    extern __shared__ __align__(16) float smem[];
    __shared__ unsigned smask[2][2];
    __shared__ int sseq[2][kTile];
    if constexpr (FIRST) {
        if (blockIdx.y == 0) scan_segment<T, N, VEC, false>(p, 0, smem, smask, sseq);
        else scan_segment<T, N, VEC, true>(p, blockIdx.y, smem, smask, sseq);
    } else {
        scan_segment<T, N, VEC, false>(p, p.nseg > 1 ? blockIdx.y + 1 : 0, smem, smask, sseq);
    }
}

// ---------------------------------------------------------------- one token
struct StepParams {
    int B, D;
    bool softplus;
    const void *x, *dt, *z, *Bm, *Cm;
    long long ldx, lddt, ldz, ldb, ldc;
    const float *A, *Dskip, *bias;
    float *S;
    void *y;
};

// N / 4 lanes per channel, four states each, SEQS sequences per thread: A is read once for all of them, and a
// state is read and written once. What is done once per (sequence, channel) is dealt out over the channel's
// lanes: lane q loads x, step and z of sequence q, forms its step size and finishes its output. Loads
// are never conditional: sequences past B and channels past D read the last one and store nothing.
template <typename T, int N, int SEQS>
__global__ void __launch_bounds__(kThreads, 8) ssm_step_kernel(StepParams p)
{
    constexpr int L = N / 4, CH = kThreads / L;
    constexpr int OWN = SEQS <= L ? 1 : SEQS / L;  // sequences a lane does the channel's work of
    constexpr int DEAL = SEQS / OWN;               // lanes that do it
    constexpr unsigned all = 0xffffffffu;
    const int tid = threadIdx.x, lane = tid & 31, q = tid % L;
    const int ncb = (p.D + CH - 1) / CH;
    const int s0 = blockIdx.x / ncb * SEQS, cc = blockIdx.x % ncb * CH + tid / L;
    const bool live = cc < p.D;
    const int c = live ? cc : p.D - 1;
    float4 h[SEQS];
    uint32_t rb[SEQS][4], rc[SEQS][4], rx[OWN], rdt[OWN], rz[OWN];
#pragma unroll
    for (int s = 0; s < SEQS; ++s) {
        const size_t seq = min(s0 + s, p.B - 1);
        h[s] = *reinterpret_cast<const float4 *>(p.S + (seq * p.D + c) * N + 4 * q);
        const T *b = static_cast<const T *>(p.Bm) + seq * p.ldb + 4 * q, *cv = static_cast<const T *>(p.Cm) + seq * p.ldc + 4 * q;
#pragma unroll
        for (int i = 0; i < 4; ++i) { rb[s][i] = load_bits(b + i); rc[s][i] = load_bits(cv + i); }
    }
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        const size_t seq = min(s0 + q % DEAL + o * DEAL, p.B - 1);
        rx[o] = load_bits(static_cast<const T *>(p.x) + seq * p.ldx + c);
        rdt[o] = load_bits(static_cast<const T *>(p.dt) + seq * p.lddt + c);
        rz[o] = p.z ? load_bits(static_cast<const T *>(p.z) + seq * p.ldz + c) : 0u;
    }
    float4 a = __ldg(reinterpret_cast<const float4 *>(p.A + (size_t)c * N + 4 * q));
    a.x = decay_rate(a.x); a.y = decay_rate(a.y); a.z = decay_rate(a.z); a.w = decay_rate(a.w);
    const float bias = p.bias ? __ldg(p.bias + c) : 0.f, skip = p.Dskip ? __ldg(p.Dskip + c) : 0.f;
    float d[OWN], x[OWN];
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        x[o] = bits_value<T>(rx[o]);
        d[o] = bits_value<T>(rdt[o]) + bias;
        if (p.softplus) d[o] = softplus(d[o]);
    }
    float part[SEQS];
#pragma unroll
    for (int s = 0; s < SEQS; ++s) {
        const int from = lane - q + s % DEAL;
        const float ds = __shfl_sync(all, d[s / DEAL], from), xs = __shfl_sync(all, x[s / DEAL], from);
        const float u = ds * xs;
        h[s].x = fmaf(decay2(ds, a.x), h[s].x, u * bits_value<T>(rb[s][0]));
        h[s].y = fmaf(decay2(ds, a.y), h[s].y, u * bits_value<T>(rb[s][1]));
        h[s].z = fmaf(decay2(ds, a.z), h[s].z, u * bits_value<T>(rb[s][2]));
        h[s].w = fmaf(decay2(ds, a.w), h[s].w, u * bits_value<T>(rb[s][3]));
        if (live && s0 + s < p.B)
            *reinterpret_cast<float4 *>(p.S + ((size_t)(s0 + s) * p.D + c) * N + 4 * q) = h[s];
        part[s] = fmaf(bits_value<T>(rc[s][0]), h[s].x, bits_value<T>(rc[s][1]) * h[s].y) +
                  fmaf(bits_value<T>(rc[s][2]), h[s].z, bits_value<T>(rc[s][3]) * h[s].w);
#pragma unroll
        for (int m = 1; m < L; m <<= 1) part[s] += __shfl_xor_sync(all, part[s], m);
    }
#pragma unroll
    for (int o = 0; o < OWN; ++o) {
        float sum = part[o * DEAL];
#pragma unroll
        for (int i = 1; i < DEAL; ++i) sum = q % DEAL == i ? part[o * DEAL + i] : sum;
        float v = fmaf(skip, x[o], sum);
        if (p.z) { const float zv = bits_value<T>(rz[o]); v *= zv * sigmoid(zv); }
        const int seq = s0 + q % DEAL + o * DEAL;
        if (live && q < DEAL && seq < p.B) store_one(static_cast<T *>(p.y) + (size_t)seq * p.D + c, v);
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
    using S = ScanShape<N>;
    const int streams = a.cu_seqlens ? 1 : a.B;
    const unsigned cb = (unsigned)((a.D + kCh - 1) / kCh);
    auto ok = [&](const void *q, long long ld) { return runs_aligned(q, ld, sizeof(T), 16); };
    const bool vec = a.D % E == 0 && ok(a.x, a.ldx) && ok(a.dt, a.lddt) && ok(a.z, a.ldz) && ok(a.y, a.D);
    auto run = [&](auto *kern, int segments) -> cudaError_t {
        const int smem = S::kFloats * (int)sizeof(float);
        const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
        kern<<<dim3(cb * streams, segments), S::kBlock, smem, st>>>(p);
        return cudaGetLastError();
    };
    if (p.nseg > 1) {
        const cudaError_t e = vec ? run(ssm_scan_kernel<T, N, true, true>, p.nseg - 1)
                                  : run(ssm_scan_kernel<T, N, false, true>, p.nseg - 1);
        if (e != cudaSuccess) return e;
    }
    const int rest = p.nseg > 1 ? p.nseg - 1 : 1;
    return vec ? run(ssm_scan_kernel<T, N, true, false>, rest) : run(ssm_scan_kernel<T, N, false, false>, rest);
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

template <typename T, int N>
cudaError_t launch_step(const StepParams &p, cudaStream_t st)
{
    // Two sequences per thread where that leaves two blocks per SM, else one, for latency. (256 sequences of 2048
    // channels, N = 16, bf16: 18.7 us with two per thread and eight blocks per SM, 18.8 to 20.7 with four and four, 22.4 with
    // one; one sequence of 1000 channels, fp32: 3.8 us with one per thread, 4.1 with four.)
    constexpr int per = kThreads / (N / 4);
    const unsigned cb = (unsigned)((p.D + per - 1) / per);
    if ((long long)((p.B + 1) / 2) * cb >= 2LL * sm_count())
        ssm_step_kernel<T, N, 2><<<(unsigned)((p.B + 1) / 2) * cb, kThreads, 0, st>>>(p);
    else
        ssm_step_kernel<T, N, 1><<<(unsigned)p.B * cb, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <typename T>
cudaError_t launch_step_n(int N, const StepParams &p, cudaStream_t st)
{
    switch (N) {
    case 8: return launch_step<T, 8>(p, st);
    case 16: return launch_step<T, 16>(p, st);
    case 32: return launch_step<T, 32>(p, st);
    default: return launch_step<T, 64>(p, st);
    }
}

}  // namespace

// Segments of the time axis. With one the scan is a single launch of a block per 32 channels; with
// g > 2 two launches of g - 1 blocks per 32 channels, each over T / g tokens. A token costs an SM that runs k blocks,
// two at a time, k units, and a block that is alone kAlone (at N = 16: 31 ns a unit, 39 ns alone; within 5% of the best of
// nine counts tried there). N = 32 and 64 run one block per SM and take the same rule, which was not measured for them.
SsmSplit ssm_scan_split(int streams, int T, int D)
{
    constexpr double kAlone = 1.27;
    const long long blocks = (long long)streams * ((D + kCh - 1) / kCh);
    const int sms = sm_count(), tiles = (T + kTile - 1) / kTile;
    auto cost = [&](int g) {
        const long long k = (blocks * (g > 1 ? g - 1 : 1) + sms - 1) / sms;
        const double per = ((tiles + g - 1) / g * (double)kTile + 64.) * (k % 2 ? k - 1 + kAlone : k);
        return g > 1 ? 2 * per + 2. * g : per;  // with a tile to fill and a tile to drain; states to compose
    };
    int best = 1;
    for (int g = 3; g <= tiles && g <= 256; ++g)
        if (cost(g) < cost(best)) best = g;
    SsmSplit s;
    s.seg = (tiles + best - 1) / best * kTile;
    if (s.seg < kTile) s.seg = kTile;
    s.nseg = (T + s.seg - 1) / s.seg;
    if (s.nseg == 2) { s.nseg = 1; s.seg = (tiles > 0 ? tiles : 1) * kTile; }
    if (s.nseg < 1) s.nseg = 1;
    return s;
}

size_t ssm_scan_workspace_bytes(int streams, int T, int D, int N)
{
    const SsmSplit s = ssm_scan_split(streams, T, D);
    if (s.nseg <= 1) return 0;
    const size_t n = (size_t)streams * s.nseg * D;
    return (n * (N + 1) * sizeof(float) + 255) / 256 * 256;
}

cudaError_t launch_ssm_scan(const SsmArgs &a, cudaStream_t st)
{
    const int streams = a.cu_seqlens ? 1 : a.B;
    if (a.T > 0 && streams > 0 && a.D > 0) {
        const SsmSplit s = ssm_scan_split(streams, a.T, a.D);
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
    return cudaSuccess;
}

cudaError_t launch_ssm_step(const SsmArgs &a, cudaStream_t st)
{
    StepParams p;
    p.B = a.B; p.D = a.D;
    p.softplus = a.softplus;
    p.x = a.x; p.dt = a.dt; p.z = a.z; p.Bm = a.Bm; p.Cm = a.Cm;
    p.ldx = a.ldx; p.lddt = a.lddt; p.ldz = a.ldz; p.ldb = a.ldb; p.ldc = a.ldc;
    p.A = a.A; p.Dskip = a.Dskip; p.bias = a.dt_bias;
    p.S = a.S_T;
    p.y = a.y;
    return a.bf16 ? launch_step_n<__nv_bfloat16>(a.N, p, st) : launch_step_n<float>(a.N, p, st);
}

}  // namespace gdr2
