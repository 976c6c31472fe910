// glr.hip -- the per-channel gated linear recurrence, forward and backward
// (include/gdn_layer.h).
//
// Forward, per sequence and channel, a_t = exp(g_t):
//   h_t = a_t h_{t-1} + x_t,   h_{-1} = h0
// Backward, lambda_t the gradient of h_t and mu_t = a_t lambda_t what it passes on:
//   lambda_t = dh_t + mu_{t+1}   (dht instead of mu_{t+1} at a sequence's last token)
//   dx_t = lambda_t,  dg_t = mu_t h_{t-1},  dh0 = mu_0
// Both are chains of affine maps s -> P s + H, bound by HBM (8 and 14 bytes per
// element in bf16 against a few operations), so each reads its tensors once:
//   - The token axis of the whole batch is cut into tiles of L tokens, one wave
//     each, C channels a lane, the tile held in registers; W tiles make a
//     segment, one workgroup.  A tile's map is composed in registers, the tiles
//     of a segment through LDS.
//   - Across segments each workgroup publishes its map (P, H) before it waits for
//     anything, then composes the maps of the segments before it.  Segments are
//     grouped by G; the last one of a group publishes the state that leaves it,
//     so a segment reads at most G - 1 maps and one state.  The order of every
//     composition is fixed by the sizes alone: equal inputs give equal bits.
//   - A sequence that begins inside takes its state from h0 and nothing from
//     before, by a branch that is uniform over the wave (a product with zero
//     would let another sequence's infinity or NaN through).
// Waiting ends: a workgroup takes its segment from a counter, so the segments
// that it waits for belong to workgroups that already run, and those publish
// their maps without waiting; a group's state waits for the previous group's
// only.  (A poll also gives up after POLLS tries and yields NaN.)
// The state is carried in fp32 throughout; h and dx are rounded once.  The
// backward recomputes h_{t-1} from the states that the forward saved at every
// tile, not from the rounded h: dg is an fp32 output.
#include "../../include/gdn_layer.h"
#include "gdr_device.hpp"
#include "layer_launch.hpp"

namespace layer {
namespace {

using gdr::bf16;
using gdr::f16;
constexpr int L = GLR_TILE;
constexpr int W = 8;            // waves (tiles) of a segment
constexpr int SEG = W * L;      // tokens of a segment
constexpr int G = 16;           // segments of a group
constexpr int PPW = (G - 2) / W + 1;   // maps a wave composes
constexpr int POLLS = 1 << 22;

template <class E, int N> struct VecU { typedef E t __attribute__((ext_vector_type(N), aligned(sizeof(E)))); };

typedef unsigned long long u64;
constexpr u64 NOT_YET = ~0ull;

// Published values are never the pattern that marks "not yet": a NaN is
// replaced by the canonical one.
__device__ __forceinline__ unsigned bits_of(float x) { return x != x ? 0x7fc00000u : __float_as_uint(x); }
__device__ __forceinline__ void publish(u64* p, float P, float H) {
    __hip_atomic_store(p, (u64)bits_of(P) << 32 | bits_of(H), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void publish(unsigned* p, float h) {
    __hip_atomic_store(p, bits_of(h), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Waits until C consecutive values are there.
template <int C> __device__ __forceinline__ void await(const u64* p, float (&P)[C], float (&H)[C]) {
    u64 v[C];
    for (int n = 0; n < POLLS; n++) {
        bool all = true;
#pragma unroll
        for (int c = 0; c < C; c++) {
            v[c] = __hip_atomic_load(p + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            all = all && v[c] != NOT_YET;
        }
        if (all) break;
        __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int c = 0; c < C; c++) P[c] = __uint_as_float(v[c] >> 32), H[c] = __uint_as_float((unsigned)v[c]);
}
template <int C> __device__ __forceinline__ void await(const unsigned* p, float (&h)[C]) {
    unsigned v[C];
    for (int n = 0; n < POLLS; n++) {
        bool all = true;
#pragma unroll
        for (int c = 0; c < C; c++) {
            v[c] = __hip_atomic_load(p + c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            all = all && v[c] != ~0u;
        }
        if (all) break;
        __builtin_amdgcn_s_sleep(1);
    }
#pragma unroll
    for (int c = 0; c < C; c++) h[c] = __uint_as_float(v[c]);
}

// ------------------------------------------------------------- sequences
// Sequence n is tokens [first(n), first(n + 1)); all values are uniform.
struct Seqs {
    const int32_t* cu;
    int T, nseq;
    __device__ __forceinline__ int first(int n) const { return cu ? cu[n] : n * T; }
    // the (non-empty) sequence of token t
    __device__ __forceinline__ int of(int t) const {
        if (!cu) return t / T;
        int lo = 0, hi = nseq;   // first(lo) <= t < first(hi)
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (cu[m] <= t) lo = m;
            else hi = m;
        }
        return lo;
    }
    // from sequence n the next one, or the one before, that has tokens
    __device__ __forceinline__ int next(int n) const {
        do n++;
        while (n + 1 < nseq && first(n + 1) == first(n));
        return n;
    }
    __device__ __forceinline__ int prev(int n) const {
        do n--;
        while (n > 0 && first(n + 1) == first(n));
        return n;
    }
};

// The tokens of a tile at which a sequence begins, as a bit mask, and the
// sequence of its first and last token.
struct Tile {
    int t0, nt;       // first token, tokens (0: past the end)
    unsigned begins;
    int n0, n1;
    __device__ __forceinline__ Tile(const Seqs& q, int t, int ntok) {
        t0 = t;
        nt = min(max(ntok - t, 0), L);
        begins = 0;
        n0 = n1 = 0;
        if (nt == 0) return;
        int n = q.of(t0);
        n0 = n;
        if (q.first(n) == t0) begins = 1;
        for (int e = q.first(n + 1); e < t0 + nt; e = q.first(n + 1)) {
            begins |= 1u << (e - t0);
            n = q.next(n);
        }
        n1 = n;
    }
};

template <int C> __device__ __forceinline__ void load_row(const float* p, float (&v)[C]) {
    const auto t = *(const typename VecU<float, C>::t*)p;
#pragma unroll
    for (int c = 0; c < C; c++) v[c] = t[c];
}
template <int C> __device__ __forceinline__ void store_row(float* p, const float (&v)[C]) {
    typename VecU<float, C>::t t;
#pragma unroll
    for (int c = 0; c < C; c++) t[c] = v[c];
    *(typename VecU<float, C>::t*)p = t;
}
// The row of sequence n of a [nseq, D] tensor, zero where it is absent.
template <int C> __device__ __forceinline__ void seq_row(const float* s, int n, int D, int ch, float (&v)[C]) {
#pragma unroll
    for (int c = 0; c < C; c++) v[c] = 0.f;
    if (s) load_row<C>(s + (long)n * D + ch, v);
}
// Sequences without tokens before token t, at which one begins (or the end of
// all): their output row is their input row.
template <int C>
__device__ __forceinline__ void pass_empty(const Seqs& q, int n, int t, const float* in, float* out, int D, int ch) {
    for (int m = n - 1; m >= 0 && q.first(m) == t; m--) {
        float v[C];
        seq_row<C>(in, m, D, ch, v);
        store_row<C>(out + (long)m * D + ch, v);
    }
}

// The workspace: a counter, the segments' maps and the groups' states, all set
// to ones before (NOT_YET; the counter then gives 0 after one increment).
struct Ws {
    unsigned* count;
    u64* map;          // [nseg][D]
    unsigned* state;   // [groups][D]: what enters group 1, 2, ...
};
constexpr size_t WS_HEAD = 256;
__host__ __device__ __forceinline__ Ws carve(void* ws, int nseg, int D) {
    char* b = (char*)ws;
    return Ws{(unsigned*)b, (u64*)(b + WS_HEAD), (unsigned*)(b + WS_HEAD + (size_t)nseg * D * 8)};
}

// What enters segment `idx` (in processing order): the composition of the maps
// of segments src .. idx - 1, src the one in which the sequence was entered, or
// the state that entered the group.  Called by all waves; `mp` holds W maps.
template <int C>
__device__ __forceinline__ void enter_segment(const Ws& ws, int idx, int src, int D, int ch, float (*mp)[2][64 * C],
                                              float (&in)[C]) {
    const int w = threadIdx.x >> 6, l = threadIdx.x & 63, g0 = idx / G * G;
    const bool whole = src >= g0;                   // the sequence was entered in this group
    const int j0 = whole ? src : g0, j = j0 + w * PPW;
    float P[C], H[C];
#pragma unroll
    for (int c = 0; c < C; c++) P[c] = 1.f, H[c] = 0.f;
    if (w == 0 && !whole) await<C>(ws.state + (size_t)(g0 / G - 1) * D + ch, H);
#pragma unroll
    for (int i = 0; i < PPW; i++) {
        if (j + i >= idx) break;
        float p[C], h[C];
        await<C>(ws.map + (size_t)(j + i) * D + ch, p, h);
        if (j + i == src) {   // whatever came before does not reach past it
#pragma unroll
            for (int c = 0; c < C; c++) P[c] = 0.f, H[c] = h[c];
        } else {
#pragma unroll
            for (int c = 0; c < C; c++) P[c] *= p[c], H[c] = p[c] * H[c] + h[c];
        }
    }
#pragma unroll
    for (int c = 0; c < C; c++) mp[w][0][l * C + c] = P[c], mp[w][1][l * C + c] = H[c];
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; c++) in[c] = mp[0][1][l * C + c];
#pragma unroll
    for (int v = 1; v < W; v++)
        if (j0 + v * PPW < idx)
#pragma unroll
            for (int c = 0; c < C; c++) in[c] = mp[v][0][l * C + c] * in[c] + mp[v][1][l * C + c];
}

// Composes the segment's tiles: `mp` the tiles' maps in processing order, bit v
// of `cut` set where tile v does not depend on what enters it.
template <int C>
__device__ __forceinline__ void through_tiles(const float (*mp)[2][64 * C], unsigned cut, int v0, int v1,
                                              float (&P)[C], float (&H)[C]) {
    const int l = threadIdx.x & 63;
    for (int v = v0; v < v1; v++) {
        if (cut >> v & 1) {
#pragma unroll
            for (int c = 0; c < C; c++) P[c] = 0.f, H[c] = mp[v][1][l * C + c];
        } else {
#pragma unroll
            for (int c = 0; c < C; c++) {
                const float p = mp[v][0][l * C + c];
                P[c] *= p;
                H[c] = p * H[c] + mp[v][1][l * C + c];
            }
        }
    }
}

// The segment's place among the others: processing index and channel block.
__device__ __forceinline__ void take(const Ws& ws, bool chain, int nblk, int* tick, int& idx, int& blk) {
    unsigned k = blockIdx.x;
    if (chain) {
        if (threadIdx.x == 0)
            *tick = (int)(__hip_atomic_fetch_add(ws.count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + 1u);
        __syncthreads();
        k = (unsigned)__builtin_amdgcn_readfirstlane(*tick);
    }
    idx = (int)(k / (unsigned)nblk);
    blk = (int)(k % (unsigned)nblk);
}

// Rows of a tile from token t0c on, C channels of each; rows past the last
// token read it again (they are not used).
template <class E, int C>
__device__ __forceinline__ void load_tile(const E* p, int D, int last, typename VecU<E, C>::t (&v)[L]) {
#pragma unroll
    for (int i = 0; i < L; i++) v[i] = *(const typename VecU<E, C>::t*)(p + (unsigned)min(i, last) * (unsigned)D);
}

template <class E, int C>
__global__ __launch_bounds__(64 * W) void glr_fwd_kernel(GlrArgs a, int nblk, int nseg, bool chain) {
    __shared__ float mp[W][2][64 * C], ep[W][2][64 * C];
    __shared__ unsigned cuts[W];
    __shared__ int tick;
    const Ws ws = carve(a.ws, nseg, a.D);
    int seg, blk;
    take(ws, chain, nblk, &tick, seg, blk);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, D = a.D;
    const int ntok = (int)a.ntok, ch = min((blk * 64 + l) * C, D - C);   // lanes past the end repeat the last channels
    const Seqs q{a.cu, a.T, a.nseq};
    const Tile tile(q, seg * SEG + w * L, ntok);
    const int t0c = min(tile.t0, ntok - 1);
    const long base = (long)t0c * D + ch;
    typename VecU<E, C>::t x[L];
    float al[L][C];
    {
        typename VecU<float, C>::t g[L];
        load_tile<float, C>(a.g + base, D, ntok - 1 - t0c, g);
        load_tile<E, C>((const E*)a.x + base, D, ntok - 1 - t0c, x);
#pragma unroll
        for (int i = 0; i < L; i++)
#pragma unroll
            for (int c = 0; c < C; c++) {   // past the end: the identity
                al[i][c] = i < tile.nt ? expf(g[i][c]) : 1.f;
                if (i >= tile.nt) x[i][c] = (E)0.f;
            }
    }
    float P[C], H[C];
#pragma unroll
    for (int c = 0; c < C; c++) P[c] = 1.f, H[c] = 0.f;
    {
        int n = tile.n0;
#pragma unroll
        for (int i = 0; i < L; i++) {
            if (tile.begins >> i & 1) {
                if (i > 0) n = q.next(n);
                seq_row<C>(a.h0, n, D, ch, H);
            }
#pragma unroll
            for (int c = 0; c < C; c++) {
                P[c] *= al[i][c];
                H[c] = al[i][c] * H[c] + (float)x[i][c];
            }
        }
    }
#pragma unroll
    for (int c = 0; c < C; c++) mp[w][0][l * C + c] = P[c], mp[w][1][l * C + c] = H[c];
    if (l == 0) cuts[w] = tile.begins != 0;
    __syncthreads();
    unsigned cut = 0;
#pragma unroll
    for (int v = 0; v < W; v++) cut |= cuts[v] << v;
    cut = __builtin_amdgcn_readfirstlane(cut);
    float in[C];
#pragma unroll
    for (int c = 0; c < C; c++) in[c] = 0.f;
    const int T0 = seg * SEG;
    if (chain) {
        if (w == 0 && seg + 1 < nseg) {
#pragma unroll
            for (int c = 0; c < C; c++) P[c] = 1.f, H[c] = 0.f;
            through_tiles<C>(mp, cut, 0, W, P, H);
#pragma unroll
            for (int c = 0; c < C; c++) publish(ws.map + (size_t)seg * D + ch + c, P[c], H[c]);
            asm volatile("" ::: "memory");   // published before anything is waited for
        }
        const int s0 = q.first(q.of(T0));   // where the sequence that enters began
        if (s0 < T0) enter_segment<C>(ws, seg, s0 / SEG, D, ch, ep, in);
        if (w == 0 && seg % G == G - 1 && seg + 1 < nseg) {
            float p1[C], out[C];
#pragma unroll
            for (int c = 0; c < C; c++) p1[c] = 1.f, out[c] = in[c];
            through_tiles<C>(mp, cut, 0, W, p1, out);
#pragma unroll
            for (int c = 0; c < C; c++) publish(ws.state + (size_t)(seg / G) * D + ch + c, out[c]);
        }
    }
    if (tile.nt == 0) return;
#pragma unroll
    for (int c = 0; c < C; c++) P[c] = 1.f;
    through_tiles<C>(mp, cut, 0, w, P, in);
    E* out = (E*)a.h + base;
    int n = tile.n0;
#pragma unroll
    for (int i = 0; i < L; i++) {
        if (tile.begins >> i & 1) {
            if (i > 0) {
                if (a.ht) store_row<C>(a.ht + (long)n * D + ch, in);   // the state that the sequence ends with
                n = q.next(n);
            }
            if (a.ht) pass_empty<C>(q, n, tile.t0 + i, a.h0, a.ht, D, ch);
            seq_row<C>(a.h0, n, D, ch, in);
        }
        if (i == 0 && a.states) store_row<C>(a.states + (long)(tile.t0 / L) * D + ch, in);
        typename VecU<E, C>::t o;
#pragma unroll
        for (int c = 0; c < C; c++) {
            in[c] = al[i][c] * in[c] + (float)x[i][c];
            o[c] = (E)in[c];
        }
        if (i < tile.nt) *(typename VecU<E, C>::t*)(out + (unsigned)i * (unsigned)D) = o;
    }
    if (a.ht && tile.t0 + tile.nt == q.first(n + 1)) {
        store_row<C>(a.ht + (long)n * D + ch, in);
        if (tile.t0 + tile.nt == ntok) pass_empty<C>(q, a.nseq, ntok, a.h0, a.ht, D, ch);
    }
}

// The segments in the reverse order of time: processing index idx is segment
// nseg - 1 - idx, tile W - 1 comes first.
template <class E, int C>
__global__ __launch_bounds__(64 * W) void glr_bwd_kernel(GlrArgs a, int nblk, int nseg, bool chain) {
    __shared__ float mp[W][2][64 * C], ep[W][2][64 * C];
    __shared__ unsigned cuts[W];
    __shared__ int tick;
    const Ws ws = carve(a.ws, nseg, a.D);
    int idx, blk;
    take(ws, chain, nblk, &tick, idx, blk);
    const int seg = nseg - 1 - idx;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 63, D = a.D;
    const int ntok = (int)a.ntok, ch = min((blk * 64 + l) * C, D - C);
    const Seqs q{a.cu, a.T, a.nseq};
    const Tile tile(q, seg * SEG + w * L, ntok);
    const int t0c = min(tile.t0, ntok - 1);
    const long base = (long)t0c * D + ch;
    // tokens that end a sequence
    unsigned ends = 0;
    if (tile.nt > 0) {
        ends = tile.begins >> 1;
        if (q.first(tile.n1 + 1) == tile.t0 + tile.nt) ends |= 1u << (tile.nt - 1);
    }
    typename VecU<E, C>::t dh[L];
    float al[L][C], hp[L][C];   // a_t and h_{t-1}
    {
        typename VecU<E, C>::t x[L];
        typename VecU<float, C>::t g[L];
        load_tile<float, C>(a.g + base, D, ntok - 1 - t0c, g);
        load_tile<E, C>((const E*)a.x + base, D, ntok - 1 - t0c, x);
        load_tile<E, C>((const E*)a.dh + base, D, ntok - 1 - t0c, dh);
        float h[C];
        load_row<C>(a.states + (long)(t0c / L) * D + ch, h);
        int n = tile.n0;
#pragma unroll
        for (int i = 0; i < L; i++) {
            if (i > 0 && (tile.begins >> i & 1)) {
                n = q.next(n);
                seq_row<C>(a.h0, n, D, ch, h);
            }
#pragma unroll
            for (int c = 0; c < C; c++) {
                al[i][c] = i < tile.nt ? expf(g[i][c]) : 1.f;   // past the end: the identity
                if (i >= tile.nt) dh[i][c] = (E)0.f;
                hp[i][c] = h[c];
                h[c] = al[i][c] * h[c] + (float)x[i][c];
            }
        }
    }
    float P[C], M[C];
#pragma unroll
    for (int c = 0; c < C; c++) P[c] = 1.f, M[c] = 0.f;
    {
        int n = tile.n1;
#pragma unroll
        for (int i = L - 1; i >= 0; i--) {
            if (ends >> i & 1) {
                if (i + 1 < tile.nt) n = q.prev(n);
                seq_row<C>(a.dht, n, D, ch, M);
            }
#pragma unroll
            for (int c = 0; c < C; c++) {
                P[c] *= al[i][c];
                M[c] = al[i][c] * ((float)dh[i][c] + M[c]);
            }
        }
    }
    const int pw = W - 1 - w;   // the tile's place in processing order
#pragma unroll
    for (int c = 0; c < C; c++) mp[pw][0][l * C + c] = P[c], mp[pw][1][l * C + c] = M[c];
    if (l == 0) cuts[pw] = ends != 0;
    __syncthreads();
    unsigned cut = 0;
#pragma unroll
    for (int v = 0; v < W; v++) cut |= cuts[v] << v;
    cut = __builtin_amdgcn_readfirstlane(cut);
    float in[C];
#pragma unroll
    for (int c = 0; c < C; c++) in[c] = 0.f;
    const int T1 = min((seg + 1) * SEG, ntok);
    if (chain) {
        if (w == 0 && seg > 0) {
#pragma unroll
            for (int c = 0; c < C; c++) P[c] = 1.f, M[c] = 0.f;
            through_tiles<C>(mp, cut, 0, W, P, M);
#pragma unroll
            for (int c = 0; c < C; c++) publish(ws.map + (size_t)idx * D + ch + c, P[c], M[c]);
            asm volatile("" ::: "memory");   // published before anything is waited for
        }
        const int e0 = q.first(q.of(T1 - 1) + 1);   // where the sequence that enters from the right ends
        if (e0 > T1) enter_segment<C>(ws, idx, nseg - 1 - (e0 - 1) / SEG, D, ch, ep, in);
        if (w == 0 && idx % G == G - 1 && seg > 0) {
            float p1[C], out[C];
#pragma unroll
            for (int c = 0; c < C; c++) p1[c] = 1.f, out[c] = in[c];
            through_tiles<C>(mp, cut, 0, W, p1, out);
#pragma unroll
            for (int c = 0; c < C; c++) publish(ws.state + (size_t)(idx / G) * D + ch + c, out[c]);
        }
    }
    if (tile.nt == 0) return;
#pragma unroll
    for (int c = 0; c < C; c++) P[c] = 1.f;
    through_tiles<C>(mp, cut, 0, pw, P, in);
    int n = tile.n1;
#pragma unroll
    for (int i = L - 1; i >= 0; i--) {
        if (ends >> i & 1) {
            if (i + 1 < tile.nt) n = q.prev(n);
            seq_row<C>(a.dht, n, D, ch, in);
        }
        typename VecU<E, C>::t o;
        float dg[C];
#pragma unroll
        for (int c = 0; c < C; c++) {
            const float lam = (float)dh[i][c] + in[c];
            in[c] = al[i][c] * lam;
            o[c] = (E)lam;
            dg[c] = in[c] * hp[i][c];
        }
        if (i < tile.nt) {
            *(typename VecU<E, C>::t*)((E*)a.dx + base + (unsigned)i * (unsigned)D) = o;
            store_row<C>(a.dg + base + (unsigned)i * (unsigned)D, dg);
        }
        if (a.dh0 && (tile.begins >> i & 1)) {
            store_row<C>(a.dh0 + (long)n * D + ch, in);
            pass_empty<C>(q, n, tile.t0 + i, a.dht, a.dh0, D, ch);
        }
    }
    if (a.dh0 && tile.t0 + tile.nt == ntok) pass_empty<C>(q, a.nseq, ntok, a.dht, a.dh0, D, ch);
}

__global__ __launch_bounds__(256) void glr_clear_kernel(uint4* p, size_t n) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) p[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

// No tokens at all: the states pass through.
__global__ __launch_bounds__(256) void glr_pass_kernel(const float* in, float* out, size_t n) {
    const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n) out[i] = in ? in[i] : 0.f;
}

int segments(const GlrArgs& a) { return (int)((a.ntok + SEG - 1) / SEG); }
// Whether a segment may begin inside a sequence.
bool chained(const GlrArgs& a) { return segments(a) > 1 && (a.cu || SEG % a.T != 0); }

hipError_t pass(const GlrArgs& a, const float* in, float* out, hipStream_t s) {
    const size_t n = (size_t)a.nseq * a.D;
    hipLaunchKernelGGL(glr_pass_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, in, out, n);
    return hipGetLastError();
}
hipError_t clear(const GlrArgs& a, hipStream_t s) {
    const size_t n = glr_ws_bytes(a) / 16;
    hipLaunchKernelGGL(glr_clear_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, (uint4*)a.ws, n);
    return hipGetLastError();
}

template <class E, int C> hipError_t run(const GlrArgs& a, bool bwd, hipStream_t s) {
    const bool chain = chained(a);
    if (chain) {
        const hipError_t e = clear(a, s);
        if (e != hipSuccess) return e;
    }
    const int nseg = segments(a), nblk = (a.D + 64 * C - 1) / (64 * C);
    const dim3 grid((unsigned)nseg * nblk), blk(64 * W);
    if (bwd) hipLaunchKernelGGL((glr_bwd_kernel<E, C>), grid, blk, 0, s, a, nblk, nseg, chain);
    else hipLaunchKernelGGL((glr_fwd_kernel<E, C>), grid, blk, 0, s, a, nblk, nseg, chain);
    return hipGetLastError();
}
template <class E> hipError_t by_width(const GlrArgs& a, bool bwd, hipStream_t s) {
    return a.D >= 4 ? run<E, 4>(a, bwd, s) : run<E, 1>(a, bwd, s);
}
hipError_t by_type(const GlrArgs& a, bool bwd, hipStream_t s) {
    switch (a.dtype) {
        case GDR_F32: return by_width<float>(a, bwd, s);
        case GDR_F16: return by_width<f16>(a, bwd, s);
        default: return by_width<bf16>(a, bwd, s);
    }
}

}  // namespace

long glr_workgroups(const GlrArgs& a) {
    const int c = a.D >= 4 ? 4 : 1;
    return (long)segments(a) * ((a.D + 64 * c - 1) / (64 * c));
}

size_t glr_ws_bytes(const GlrArgs& a) {
    if (a.ntok == 0 || !chained(a)) return 0;
    const int nseg = segments(a);
    const size_t b = WS_HEAD + (size_t)nseg * a.D * 8 + (size_t)((nseg + G - 1) / G) * a.D * 4;
    return (b + 15) & ~(size_t)15;
}

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t s) {
    return a.ntok == 0 ? pass(a, a.h0, a.ht, s) : by_type(a, false, s);
}
hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t s) {
    return a.ntok == 0 ? pass(a, a.dht, a.dh0, s) : by_type(a, true, s);
}

}  // namespace layer
