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
//     segment, one pass of a workgroup.  A tile's map is composed in registers,
//     the tiles of a segment through LDS.
//   - Across segments: a workgroup publishes its segment's map (P, H) before it
//     waits for anything.  G segments make a group, whose last one publishes the
//     group's map; G groups make a block, whose last one publishes the state that
//     leaves it.  What enters a segment is one state, at most G - 1 group maps and
//     at most G - 1 maps, one read by each wave, composed in an order fixed by
//     the sizes alone: equal inputs give equal bits.
//   - A sequence that begins inside takes its state from h0 and nothing from
//     before, by a branch that is uniform over the wave (a product with zero
//     would let another sequence's infinity or NaN through).
// Waiting ends, whatever the order in which workgroups start: after `polls` tries
// a workgroup takes up the first earlier segment that still owes a word of its own
// (its map, its group's, its block's state), as if it were its own (both give the
// same bits), and then begins its own again.  The first segment that is not finished
// waits for nothing, so it is finished by whoever has it, or by one that waits for
// it.  The rule is in glr_chain.hpp.
// A product P of gates may overflow where the state itself would not, if gates
// above 1 follow one another (include/gdn_layer.h bounds them); where it
// underflows, what it multiplies is lost too.
// Measured (bf16, D = 2048): one sequence of 32768 tokens 111 us forward and 6 to
// clear the words, 4.6 TB/s of the 537 MB that it needs; 94 to 100 us with segments
// that do not wait for one another (wrong results, the same traffic), so a fifth of
// the time is the exchange: some 6 of the 17 us that a workgroup lives, two hops of
// 3.5 us from one workgroup's store to another's load.  Forward and backward of
// twelve sequences, 65536 tokens: 603 us (229 and 362, 11 to clear; 4.9 TB/s).
// Tried, per step: whole rows polled instead of one element 136 against 126 us; 8
// tiles a segment against 12, 126 against 118 us; a counter handing out segments (so that no workgroup could
// wait for one that has not started) 6 to 8 % more, one per channel block 705
// against 595 us forward and backward, since the blocks' rows then drift apart in
// time; four channels a lane 190 against 140 us (154 registers, one workgroup a CU).
// Registers: 80 a lane in the 16-bit forward of two channels a lane, whose bf16
// instance spills one value more (8 bytes a lane); 36 to 70 uniform values of every kernel are
// kept in lanes of vector registers.
// The state is carried in fp32 throughout; h and dx are rounded once.  The
// backward recomputes h_{t-1} from the states that the forward saved at every
// tile, not from the rounded h: dg is an fp32 output.
#include "../../include/gdn_layer.h"
#include "gdr_device.hpp"
#include "glr_chain.hpp"
#include "layer_launch.hpp"

namespace layer {
namespace {

using chain::G;
using gdr::bf16;
using gdr::f16;
constexpr int L = GLR_TILE;
constexpr int SLEEP = 8;        // 64 clocks each between two looks

template <class E, int N> struct VecU { typedef E t __attribute__((ext_vector_type(N), aligned(sizeof(E)))); };

typedef unsigned long long u64;
constexpr u64 NOT_YET = ~0ull;

// Published values are never the pattern that marks "not yet": a NaN is
// replaced by the canonical one.
__device__ __forceinline__ unsigned bits_of(float x) { return x != x ? 0x7fc00000u : __float_as_uint(x); }
__device__ __forceinline__ void publish(u64* p, float P, float H) {
    __hip_atomic_store(p, (u64)bits_of(P) << 32 | bits_of(H), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ u64 peek(const u64* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ------------------------------------------------------------- sequences
// Sequence n is tokens [first(n), first(n + 1)); all values are uniform.  What
// the device's cu_seqlens holds is kept within the tokens and sequences there
// are, so that a copy that differs from the host's gives wrong results and not
// accesses out of bounds.
struct Seqs {
    const int32_t* cu;
    int T, nseq, ntok;
    __device__ __forceinline__ int first(int n) const {
        return cu ? min(max(__builtin_amdgcn_readfirstlane(cu[n]), 0), ntok) : n * T;
    }
    // the (non-empty) sequence of token t
    __device__ __forceinline__ int of(int t) const {
        if (!cu) return t / T;
        int lo = 0, hi = nseq;   // first(lo) <= t < first(hi)
        while (hi - lo > 1) {
            const int m = (lo + hi) >> 1;
            if (first(m) <= t) lo = m;
            else hi = m;
        }
        return lo;
    }
    // from sequence n the next one, or the one before, that has tokens
    __device__ __forceinline__ int next(int n) const {
        while (++n + 1 < nseq && first(n + 1) == first(n)) {
        }
        return min(n, nseq - 1);
    }
    __device__ __forceinline__ int prev(int n) const {
        while (--n > 0 && first(n + 1) == first(n)) {
        }
        return max(n, 0);
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
        for (int e = q.first(n + 1); n + 1 < q.nseq && e < t0 + nt; e = q.first(n + 1)) {
            begins |= 1u << ((e - t0) & 31);
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
template <int C> __device__ __forceinline__ void seq_row(const float* s, int n, int D, unsigned ch, float (&v)[C]) {
#pragma unroll
    for (int c = 0; c < C; c++) v[c] = 0.f;
    if (s) load_row<C>(gdr::at32(s + (long)n * D, ch), v);
}
// Sequences without tokens before token t, at which one begins (or the end of
// all): their output row is their input row.
template <int C>
__device__ __forceinline__ void pass_empty(const Seqs& q, int n, int t, const float* in, float* out, int D,
                                           unsigned ch) {
    for (int m = n - 1; m >= 0 && q.first(m) == t; m--) {
        float v[C];
        seq_row<C>(in, m, D, ch, v);
        store_row<C>(gdr::at32(out + (long)m * D, ch), v);
    }
}

// The workspace: the maps of segments and groups and the states that leave blocks
// (as maps with P = 0), all set to NOT_YET before.
struct Ws {
    u64 *map, *group, *state;   // [segments][D], [groups][D], [blocks][D]
};
__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }
__host__ __device__ __forceinline__ size_t ws_bytes(int nseg, int D) {
    return ((size_t)nseg + ceil_div(nseg, G) + ceil_div(nseg, G * G)) * D * 8;
}
__device__ __forceinline__ Ws carve(void* ws, int nseg, int D) {
    u64* group = (u64*)ws + (size_t)nseg * D;
    return Ws{(u64*)ws, group, group + (size_t)ceil_div(nseg, G) * D};
}

// Composes onto (P, H) the tiles [v0, v1) of a segment: `mp` their maps in
// processing order, bit v of `cut` set where tile v does not depend on what enters it.
template <int C>
__device__ __forceinline__ void through_tiles(const float (*mp)[2][64 * C], unsigned cut, int v0, int v1,
                                              float (&P)[C], float (&H)[C]) {
    const int l = gdr::lane_o();
#pragma unroll 2
    for (int v = v0; v < v1; v++) {
        const bool cuts = cut >> v & 1;
#pragma unroll
        for (int c = 0; c < C; c++) {
            const float p = mp[v][0][l * C + c], h = mp[v][1][l * C + c];
            P[c] = cuts ? 0.f : P[c] * p;
            H[c] = cuts ? h : p * H[c] + h;
        }
    }
}

// Bit v: tile v of the segment does not depend on what enters it.
template <int W> __device__ __forceinline__ unsigned cut_bits(const unsigned* cuts) {
    unsigned all = 0;
#pragma unroll
    for (int v = 0; v < W; v++) all |= cuts[v] << v;
    return __builtin_amdgcn_readfirstlane(all);
}
template <int W, int C> using Maps = float[W][2][64 * C];

// Hands a wave's tile map (P, H) to the others and composes the maps of the tiles
// before its own (kept in `qi` for enter_tile), and its own onto them into (P, H).
// `cut`: the tile does not depend on what enters it.  Returns whether (P, H) so
// composed does not.
template <int W, int C>
__device__ __forceinline__ bool tiles_before(Maps<W, C>& mp, Maps<W, C>& qi, unsigned* cuts, int w, bool cut,
                                             float (&P)[C], float (&H)[C]) {
    const int l = gdr::lane_o();
#pragma unroll
    for (int c = 0; c < C; c++) mp[w][0][l * C + c] = P[c], mp[w][1][l * C + c] = H[c];
    if (l == 0) cuts[w] = cut;
    gdr::lds_barrier();
    const unsigned all = cut_bits<W>(cuts);
    float Q[C], I[C];
#pragma unroll
    for (int c = 0; c < C; c++) Q[c] = 1.f, I[c] = 0.f;
    through_tiles<C>(mp, all, 0, w, Q, I);
#pragma unroll
    for (int c = 0; c < C; c++) {
        qi[w][0][l * C + c] = Q[c], qi[w][1][l * C + c] = I[c];
        H[c] = cut ? H[c] : P[c] * I[c] + H[c];
        P[c] = cut ? 0.f : P[c] * Q[c];
    }
    return all & ((2u << w) - 1);
}
// What enters a tile: the maps of those before it applied to what enters the segment.
template <int W, int C>
__device__ __forceinline__ void enter_tile(const Maps<W, C>& qi, unsigned cuts_before, int w, float (&in)[C]) {
    const int l = gdr::lane_o();
#pragma unroll
    for (int c = 0; c < C; c++) {
        const float I = qi[w][1][l * C + c];
        in[c] = cuts_before ? I : qi[w][0][l * C + c] * in[c] + I;
    }
}

// Waits until the maps at `a` and `b` (uniform; NULL: none) are there and leaves
// them in LDS.  Both are read at once, so what is there costs one round trip; what
// is not is looked for by one element of each (whole rows read by every wave in
// flight over and over would take a good part of the bandwidth), then read again.
// False after `polls` tries without success.
template <int W, int C>
__device__ __forceinline__ bool await(const u64* a, const u64* b, unsigned ch, int w, int polls, Maps<W, C>& ea,
                                      Maps<W, C>& eb) {
    u64 u[C], v[C];
    bool all = false;
    const unsigned one = __builtin_amdgcn_readfirstlane(ch) + C - 1;
    for (int n = 0;;) {
#pragma unroll
        for (int c = 0; c < C; c++) {
            if (a) u[c] = peek(gdr::at32(a, ch + c));
            if (b) v[c] = peek(gdr::at32(b, ch + c));
        }
        all = true;
#pragma unroll
        for (int c = 0; c < C; c++) all = all && (!a || u[c] != NOT_YET) && (!b || v[c] != NOT_YET);
        all = __all(all);
        if (all || ++n >= polls) break;
        for (; n < polls; n++) {
            __builtin_amdgcn_s_sleep(SLEEP);
            const u64 x = a ? peek(a + one) : 0, y = b ? peek(b + one) : 0;
            if (x != NOT_YET && y != NOT_YET) break;
        }
    }
    const int l = gdr::lane_o();
#pragma unroll
    for (int c = 0; c < C; c++) {
        const int i = l * C + c;
        if (a) ea[w][0][i] = __uint_as_float((unsigned)(u[c] >> 32)), ea[w][1][i] = __uint_as_float((unsigned)u[c]);
        if (b) eb[w][0][i] = __uint_as_float((unsigned)(v[c] >> 32)), eb[w][1][i] = __uint_as_float((unsigned)v[c]);
    }
    return all;
}

// Whether all waves of the workgroup say yes, after a barrier.
template <int W> __device__ __forceinline__ bool all_waves(bool yes, unsigned* votes, int w) {
    if (gdr::lane_o() == 0) votes[w] = yes;
    gdr::lds_barrier();
    unsigned all = 1;
#pragma unroll
    for (int v = 0; v < W; v++) all &= votes[v];
    return __builtin_amdgcn_readfirstlane(all);
}

template <int C>
__device__ __forceinline__ void publish_row(u64* p, unsigned ch, const float (&P)[C], const float (&H)[C]) {
#pragma unroll
    for (int c = 0; c < C; c++) publish(gdr::at32(p, ch + c), P[c], H[c]);
    asm volatile("" ::: "memory");   // published before anything after it is waited for
}

// All of a segment's business with the others, by all waves: publishes its map,
// its group's and its block's state where it is their last, and returns what
// enters it.  `idx` counts segments in processing order, `src` is the one in which
// the sequence that enters was itself entered (src = idx: none enters).  (P, H) is
// the segment's map in wave W - 1 (w: place in processing order), `cut` whether it
// does not depend on what enters; `tot` keeps it.  False if it did not get all
// that it waits for.
template <int W, int C>
__device__ __forceinline__ bool exchange(const Ws& ws, int idx, int nseg, int src, int D, unsigned ch, int w, int polls,
                                         bool cut, const float (&P)[C], const float (&H)[C], Maps<W, C>& ea,
                                         Maps<W, C>& eb, float (*tot)[64 * C], unsigned (*votes)[W],
                                         float (&in)[C]) {
    const int l = gdr::lane_o(), g = idx / G;
    const bool later = idx + 1 < nseg, tells = w == W - 1 && later, closes = later && chain::closes_group(idx);
    const auto [first, na, gfirst, nb, outside, far] = chain::reads(idx, src);
    const u64* a = w < na ? ws.map + (size_t)(first + w) * D : nullptr;
    const u64* b = w >= nb ? nullptr : far && w == 0 ? ws.state + (size_t)(g / G - 1) * D
                                                     : ws.group + (size_t)(gfirst + w - far) * D;
    if (tells) {
        publish_row<C>(ws.map + (size_t)idx * D, ch, P, H);
        if (closes)
#pragma unroll
            for (int c = 0; c < C; c++) tot[0][l * C + c] = P[c], tot[1][l * C + c] = H[c];
    }
    if (closes) {   // the group's map needs the maps of the group only
        float p[C], h[C];
#pragma unroll
        for (int c = 0; c < C; c++) p[c] = 1.f, h[c] = 0.f;
        if (na > 0) {
            if (!all_waves<W>(await<W, C>(a, nullptr, ch, w, polls, ea, eb), votes[0], w)) return false;
            through_tiles<C>(ea, outside ? 0u : 1u, 0, na, p, h);
        }
        if (tells) {
#pragma unroll
            for (int c = 0; c < C; c++) {
                const float P1 = tot[0][l * C + c], H1 = tot[1][l * C + c];
                p[c] = cut ? 0.f : P1 * p[c];
                h[c] = cut ? H1 : P1 * h[c] + H1;
            }
            publish_row<C>(ws.group + (size_t)g * D, ch, p, h);
        }
        a = nullptr;
    }
    if (src < idx) {
        if (!all_waves<W>(await<W, C>(a, b, ch, w, polls, ea, eb), votes[1], w)) return false;
        float p[C];
#pragma unroll
        for (int c = 0; c < C; c++) p[c] = 1.f, in[c] = 0.f;
        through_tiles<C>(eb, far ? 0u : 1u, 0, nb, p, in);
        through_tiles<C>(ea, outside ? 0u : 1u, 0, na, p, in);
    }
    if (tells && chain::closes_block(idx)) {
        float p[C], h[C];
#pragma unroll
        for (int c = 0; c < C; c++) {
            const float P1 = tot[0][l * C + c], H1 = tot[1][l * C + c];
            p[c] = 0.f;
            h[c] = cut ? H1 : P1 * in[c] + H1;
        }
        publish_row<C>(ws.state + (size_t)(g / G) * D, ch, p, h);
    }
    return true;
}

// The first segment before `idx` that still owes a word (idx: none), found by the
// first wave for all.
template <int C>
__device__ __forceinline__ int first_unfinished(const Ws& ws, int idx, int D, unsigned ch, int w, int& found) {
    const auto there = [&](const u64* rows, int j) {
        bool yes = true;
#pragma unroll
        for (int c = 0; c < C; c++) yes = yes && peek(gdr::at32(rows + (size_t)j * D, ch + c)) != NOT_YET;
        return (bool)__all(yes);
    };
    if (w == 0) {
        const int j = chain::first_unfinished(
            idx, [&](int i) { return there(ws.map, i); }, [&](int i) { return there(ws.group, i); },
            [&](int i) { return there(ws.state, i); });
        if (threadIdx.x == 0) found = j;
    }
    gdr::lds_barrier();
    return __builtin_amdgcn_readfirstlane(found);
}

// exp(g), off by at most (|g| + 3) 2^-24 of itself: the exponent's one rounding,
// |g| 2^-24, and one unit in the last place, 2 2^-24, for exp2 (log2(e) in two
// parts: its one-part rounding alone adds 0.22 |g|); zero below 2^-126.  (expf is
// within 2 2^-24 at some ten operations instead of three.)  Where g is large the
// state hardly passes on; where it is small, the state that passes n tokens is off
// by up to 2 n 2^-24 of itself from the gates' last places, as any gate held in
// fp32 is by a part of that.
__device__ __forceinline__ float gate(float g) {
    return __builtin_amdgcn_exp2f(__builtin_fmaf(g, 0x1.715476p+0f, g * 0x1.4ae0cp-26f));
}

// Keeps a value as it was loaded: its widening to fp32 is not carried from one
// pass over the tile to the next in twice the registers.
template <class E, int C> __device__ __forceinline__ void as_loaded(typename VecU<E, C>::t (&v)[L]) {
    if constexpr (C * sizeof(E) >= 4) {
        constexpr int N = C * sizeof(E) / 4;
#pragma unroll
        for (int i = 0; i < L; i++) {
            unsigned u[N];
            __builtin_memcpy(u, &v[i], 4 * N);
#pragma unroll
            for (int k = 0; k < N; k++) asm volatile("" : "+v"(u[k]));
            __builtin_memcpy(&v[i], u, 4 * N);
        }
    }
}

// A lane's first channel; lanes past the end repeat the last ones.  (lane_o: what
// derives from the lane is formed where it is used, not held over the kernel's loop.)
template <int C> __device__ __forceinline__ unsigned channel(int blk, int D) {
    return (unsigned)min((blk * 64 + gdr::lane_o()) * C, D - C);
}

// Tokens past the last one are the identity.
template <class E, int C>
__device__ __forceinline__ void past_end(float (&al)[L][C], typename VecU<E, C>::t (&v)[L], int nt) {
#pragma unroll
    for (int i = 0; i < L; i++)
        if (i >= nt)
#pragma unroll
            for (int c = 0; c < C; c++) al[i][c] = 1.f, v[i][c] = (E)0.f;
}

// The same value, tested anew: conditions on it that are uniform are not kept
// as one 64-bit mask each from one pass over the tile to the next.
template <class T> __device__ __forceinline__ T anew(T x) {
    asm volatile("" : "+s"(x));
    return x;
}

// Rows of a tile, C channels from `ch` of each; rows past the last token read it
// again (they are not used).  The row bases are uniform, a lane's channel is a
// 32-bit offset.  Every element is read and written once: non-temporal.
template <class E, int C>
__device__ __forceinline__ void load_tile(const E* p, int D, int last, unsigned ch, typename VecU<E, C>::t (&v)[L]) {
#pragma unroll
    for (int i = 0; i < L; i++) {
        v[i] = __builtin_nontemporal_load((const typename VecU<E, C>::t*)gdr::at32(p, ch));
        p += i < last ? D : 0;
    }
}
template <class E, int C>
__device__ __forceinline__ void store_nt(E* row, unsigned ch, typename VecU<E, C>::t v) {
    __builtin_nontemporal_store(v, (typename VecU<E, C>::t*)gdr::at32(row, ch));
}

template <class E, int C, int W>
__global__ __launch_bounds__(64 * W, sizeof(E) == 4 ? 4 : 6) void glr_fwd_kernel(GlrArgs a, int nblk, int nseg,
                                                                               bool chain) {
    static_assert(G <= W, "one wave reads one map of a row");
    constexpr int SEG = W * L;   // tokens of a segment
    __shared__ Maps<W, C> mp, ea, eb, qi;
    __shared__ float tot[2][64 * C];
    __shared__ unsigned cuts[W], votes[2][W];
    __shared__ int missing;
    const Ws ws = carve(a.ws, nseg, a.D);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), D = a.D;
    const int ntok = (int)a.ntok;
    const Seqs q{a.cu, a.T, a.nseq, ntok};
    const int own = blockIdx.x / nblk, blk = blockIdx.x % nblk;
    for (int seg = own;;) {
        const unsigned ch = channel<C>(blk, D);
        const Tile tile(q, seg * SEG + w * L, ntok);
        const int t0c = min(tile.t0, ntok - 1), T0 = seg * SEG;
        const long base = (long)t0c * D;
        typename VecU<E, C>::t x[L];
        float al[L][C];
        {
            typename VecU<float, C>::t g[L];
            load_tile<float, C>(a.g + base, D, ntok - 1 - t0c, ch, g);
            load_tile<E, C>((const E*)a.x + base, D, ntok - 1 - t0c, ch, x);
#pragma unroll
            for (int i = 0; i < L; i++)
#pragma unroll
                for (int c = 0; c < C; c++) al[i][c] = gate(g[i][c]);
            if (tile.nt < L) past_end<E, C>(al, x, tile.nt);
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
        float in[C];   // what enters the segment
        const bool cut = tiles_before<W, C>(mp, qi, cuts, w, tile.begins != 0, P, H);
#pragma unroll
        for (int c = 0; c < C; c++) in[c] = 0.f;
        bool got = true;
        if (chain) {
            const int s0 = q.first(q.of(T0));   // where the sequence that enters began
            const int from = s0 < T0 ? s0 / SEG : seg;
            got = exchange<W, C>(ws, seg, nseg, from, D, ch, w, a.polls, cut, P, H, ea, eb, tot, votes, in);
        }
        if (got && tile.nt > 0) {
            as_loaded<E, C>(x);
            const unsigned begins = anew(tile.begins);
            const int nt = anew(tile.nt);
            enter_tile<W, C>(qi, cut_bits<W>(cuts) & ((1u << w) - 1), w, in);
            int n = tile.n0;
            E* out = (E*)a.h + base;
#pragma unroll
            for (int i = 0; i < L; i++, out += D) {
                if (begins >> i & 1) {
                    if (i > 0) {
                        // the state that the sequence ends with
                        if (a.ht) store_row<C>(gdr::at32(a.ht + (long)n * D, ch), in);
                        n = q.next(n);
                    }
                    if (a.ht) pass_empty<C>(q, n, tile.t0 + i, a.h0, a.ht, D, ch);
                    seq_row<C>(a.h0, n, D, ch, in);
                }
                if (i == 0 && a.states) store_row<C>(gdr::at32(a.states + (long)(tile.t0 / L) * D, ch), in);
                typename VecU<E, C>::t o;
#pragma unroll
                for (int c = 0; c < C; c++) {
                    in[c] = al[i][c] * in[c] + (float)x[i][c];
                    o[c] = (E)in[c];
                }
                if (i < nt) store_nt<E, C>(out, ch, o);
            }
            if (a.ht && tile.t0 + tile.nt == q.first(n + 1)) {
                store_row<C>(gdr::at32(a.ht + (long)n * D, ch), in);
                if (tile.t0 + tile.nt == ntok) pass_empty<C>(q, a.nseq, ntok, a.h0, a.ht, D, ch);
            }
        }
        if (got && seg == own) return;
        gdr::lds_barrier();   // what the next pass writes to LDS has been read
        seg = got ? own : first_unfinished<C>(ws, own, D, ch, w, missing);
    }
}

// The segments in the reverse order of time: processing index idx is segment
// nseg - 1 - idx, tile W - 1 comes first.
template <class E, int C, int W>
__global__ __launch_bounds__(64 * W, 4) void glr_bwd_kernel(GlrArgs a, int nblk, int nseg, bool chain) {
    static_assert(G <= W, "one wave reads one map of a row");
    constexpr int SEG = W * L;   // tokens of a segment
    __shared__ Maps<W, C> mp, ea, eb, qi;
    __shared__ float tot[2][64 * C];
    __shared__ unsigned cuts[W], votes[2][W];
    __shared__ int missing;
    const Ws ws = carve(a.ws, nseg, a.D);
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), D = a.D;
    const int ntok = (int)a.ntok, pw = W - 1 - w;   // pw: the tile's place in processing order
    const Seqs q{a.cu, a.T, a.nseq, ntok};
    const int own = blockIdx.x / nblk, blk = blockIdx.x % nblk;
    for (int idx = own;;) {
        const int seg = nseg - 1 - idx;
        const unsigned ch = channel<C>(blk, D);
        const Tile tile(q, seg * SEG + w * L, ntok);
        const int t0c = min(tile.t0, ntok - 1), T1 = min((seg + 1) * SEG, ntok);
        const long base = (long)t0c * D;
        unsigned ends = 0;   // tokens that end a sequence
        if (tile.nt > 0) {
            ends = tile.begins >> 1;
            if (q.first(tile.n1 + 1) == tile.t0 + tile.nt) ends |= 1u << (tile.nt - 1);
        }
        typename VecU<E, C>::t dh[L];
        float al[L][C], hp[L][C];   // a_t and h_{t-1}
        {
            typename VecU<E, C>::t x[L];
            typename VecU<float, C>::t g[L];
            load_tile<float, C>(a.g + base, D, ntok - 1 - t0c, ch, g);
            load_tile<E, C>((const E*)a.x + base, D, ntok - 1 - t0c, ch, x);
            load_tile<E, C>((const E*)a.dh + base, D, ntok - 1 - t0c, ch, dh);
            float h[C];
            load_row<C>(gdr::at32(a.states + (long)(t0c / L) * D, ch), h);
#pragma unroll
            for (int i = 0; i < L; i++)
#pragma unroll
                for (int c = 0; c < C; c++) al[i][c] = gate(g[i][c]);
            if (tile.nt < L) past_end<E, C>(al, dh, tile.nt);
            int n = tile.n0;
#pragma unroll
            for (int i = 0; i < L; i++) {
                if (i > 0 && (tile.begins >> i & 1)) {
                    n = q.next(n);
                    seq_row<C>(a.h0, n, D, ch, h);
                }
#pragma unroll
                for (int c = 0; c < C; c++) {
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
        float in[C];
        const bool cut = tiles_before<W, C>(mp, qi, cuts, pw, ends != 0, P, M);
#pragma unroll
        for (int c = 0; c < C; c++) in[c] = 0.f;
        bool got = true;
        if (chain) {
            const int e0 = q.first(q.of(T1 - 1) + 1);   // where the sequence that enters from the right ends
            const int from = e0 > T1 ? nseg - 1 - (e0 - 1) / SEG : idx;
            got = exchange<W, C>(ws, idx, nseg, from, D, ch, pw, a.polls, cut, P, M, ea, eb, tot, votes, in);
        }
        if (got && tile.nt > 0) {
            as_loaded<E, C>(dh);
            const unsigned begins = anew(tile.begins), end = anew(ends);
            const int nt = anew(tile.nt);
            enter_tile<W, C>(qi, cut_bits<W>(cuts) & ((1u << pw) - 1), pw, in);
            int n = tile.n1;
            E* dx = (E*)a.dx + base + (long)(L - 1) * D;
            float* dgr = a.dg + base + (long)(L - 1) * D;
#pragma unroll
            for (int i = L - 1; i >= 0; i--, dx -= D, dgr -= D) {
                if (end >> i & 1) {
                    if (i + 1 < nt) n = q.prev(n);
                    seq_row<C>(a.dht, n, D, ch, in);
                }
                typename VecU<E, C>::t o;
                typename VecU<float, C>::t dg;
#pragma unroll
                for (int c = 0; c < C; c++) {
                    const float lam = (float)dh[i][c] + in[c];
                    in[c] = al[i][c] * lam;
                    o[c] = (E)lam;
                    dg[c] = in[c] * hp[i][c];
                }
                if (i < nt) {
                    store_nt<E, C>(dx, ch, o);
                    store_nt<float, C>(dgr, ch, dg);
                }
                if (a.dh0 && (begins >> i & 1)) {
                    store_row<C>(gdr::at32(a.dh0 + (long)n * D, ch), in);
                    pass_empty<C>(q, n, tile.t0 + i, a.dht, a.dh0, D, ch);
                }
            }
            if (a.dh0 && tile.t0 + tile.nt == ntok) pass_empty<C>(q, a.nseq, ntok, a.dht, a.dh0, D, ch);
        }
        if (got && idx == own) return;
        gdr::lds_barrier();   // what the next pass writes to LDS has been read
        idx = got ? own : first_unfinished<C>(ws, own, D, ch, w, missing);
    }
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

// Channels of a lane: two, but one where a wave then covers the row alone.
int width(const GlrArgs& a) { return a.D > 64 ? 2 : 1; }
// Tiles of a segment.  More of them make fewer segments wait for one another, but
// a workgroup needs its waves at once: two workgroups of 12 waves fill what the
// forward's 80 registers a lane leave (fp32 x takes 16 more: 8 waves), two of 8
// the backward's 116.
constexpr int WF = 12, WF32 = 8, WB = 8;
int tiles_of(const GlrArgs& a, bool bwd) { return bwd ? WB : a.dtype == GDR_F32 ? WF32 : WF; }

int segments(const GlrArgs& a, int w) { return (int)((a.ntok + w * L - 1) / (w * L)); }
int blocks(const GlrArgs& a) {
    const int c = 64 * width(a);
    return (a.D + c - 1) / c;
}
// Whether a segment of w tiles may begin inside a sequence.
bool chained(const GlrArgs& a, int w) { return segments(a, w) > 1 && (a.cu || w * L % a.T != 0); }
size_t ws_of(const GlrArgs& a, int w) {
    return chained(a, w) ? (ws_bytes(segments(a, w), a.D) + 15) & ~(size_t)15 : 0;
}

hipError_t pass(const GlrArgs& a, const float* in, float* out, hipStream_t s) {
    const size_t n = (size_t)a.nseq * a.D;
    hipLaunchKernelGGL(glr_pass_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, in, out, n);
    return hipGetLastError();
}

template <class E, int C> hipError_t run(const GlrArgs& a, bool bwd, hipStream_t s) {
    const int w = tiles_of(a, bwd), nseg = segments(a, w), nblk = blocks(a);
    const bool chain = chained(a, w);
    if (chain) {
        const size_t n = ws_of(a, w) / 16;
        hipLaunchKernelGGL(glr_clear_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, s, (uint4*)a.ws, n);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    const dim3 grid((unsigned)nseg * nblk), blk(64 * w);
    if (bwd) hipLaunchKernelGGL((glr_bwd_kernel<E, C, WB>), grid, blk, 0, s, a, nblk, nseg, chain);
    else hipLaunchKernelGGL((glr_fwd_kernel<E, C, sizeof(E) == 4 ? WF32 : WF>), grid, blk, 0, s, a, nblk, nseg, chain);
    return hipGetLastError();
}
template <class E> hipError_t by_width(const GlrArgs& a, bool bwd, hipStream_t s) {
    return width(a) == 2 ? run<E, 2>(a, bwd, s) : run<E, 1>(a, bwd, s);
}
hipError_t by_type(const GlrArgs& a, bool bwd, hipStream_t s) {
    switch (a.dtype) {
        case GDR_F32: return by_width<float>(a, bwd, s);
        case GDR_F16: return by_width<f16>(a, bwd, s);
        default: return by_width<bf16>(a, bwd, s);
    }
}

}  // namespace

long glr_threads(const GlrArgs& a) {
    const int wf = tiles_of(a, false), wb = tiles_of(a, true);
    const long f = (long)segments(a, wf) * wf, b = (long)segments(a, wb) * wb;
    return 64 * (f > b ? f : b) * blocks(a);
}

size_t glr_ws_bytes(const GlrArgs& a) {
    if (a.ntok == 0) return 0;
    const size_t f = ws_of(a, tiles_of(a, false)), b = ws_of(a, tiles_of(a, true));
    return f > b ? f : b;
}

hipError_t launch_glr_fwd(const GlrArgs& a, hipStream_t s) {
    return a.ntok == 0 ? pass(a, a.h0, a.ht, s) : by_type(a, false, s);
}
hipError_t launch_glr_bwd(const GlrArgs& a, hipStream_t s) {
    return a.ntok == 0 ? pass(a, a.dht, a.dh0, s) : by_type(a, true, s);
}

}  // namespace layer
