// la_scan.cu -- the gated linear recurrence, elementwise per (sequence, head,
// channel):
//     s_t = exp(g_t) s_{t-1} + x_t,   o_t = s_t
// and its backward.  With K_t = exp(g_t) G_t, G_t = dL/ds_t:
//     G_t = do_t + K_{t+1},   dx_t = G_t,   dg_t = K_t s_{t-1},
// K after the last token being the final state's gradient, K at the first
// token the initial state's.
//
// Both are chains of maps s -> A s + B, which compose:
//     (A2, B2) o (A1, B1) = (A2 A1, A2 B1 + B2).
// So a team of threads takes a tile of SCAN_TILE tokens of a sequence x CT
// channels at once: its token groups compose their L tokens, the groups are
// composed through shared memory, and the state then goes through the tokens
// again.  Teams walk along a sequence, tile by tile, with the state in registers;
// x, g (and do) are read once and o (dx, dg) written once.
// A CTA per SM: a warp has the teams' tiles copied to a ring of stages by TMA, so
// that copies are under way at all times.
//
// A tile takes a team 1.8 us (backward 2.8) however fast its data come.  Where
// there are fewer sequences x channels than teams, two or four teams of a CTA take
// the tiles of a chain in turn, and only the step from the state before a tile to
// the one after it goes from team to team (1.1 us a tile with four, 128 chains of
// 64 tiles: 68 us, 116 with one; backward, with two: 134 and 183).
// Where there are fewer still, the sequences are cut into segments: a first pass
// composes each segment's map s -> A s + B (it reads the inputs and writes nothing
// else), and a segment starts from the maps of those before it.  That pass adds
// 2/3 of the reads; the alternative, tiles that wait for the state of the tile
// before them in another CTA, measured 143 us against 108 (b1 h8 d128 n65536
// forward): every tile of the GPU then waits at once, two to four microseconds a
// round.
//
// Short sequences (a few tokens of many rows, decoding) take a thread per four
// channels, which walks its sequence alone (serial, below).
//
// Bound: HBM, 6 (bf16 gate) or 8 bytes a value forward, 10 or 14 backward, and
// close to it the issue rate: 20 instructions a value forward, 38 backward, half
// of the issue slots.  bf16, b4 h32 d128 n8192 (134 M values): forward 128 us, 0.93
// of HBM's rate, backward 242 us, 0.82.  In segments (b1 h8 n262144, 268 M):
// forward 408 us, 0.58 (0.97 of the 10 bytes that it moves), backward 673, 0.59.
// Segments and teams are chosen by the number of sequences, not by their lengths:
// one of 262144 tokens beside 64 of one token is not cut (forward 3.5 ms).

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include "../../include/la.h"
#include "la_f32x2.cuh"
#include "la_internal.h"
#include "la_sm100.cuh"

namespace la {
namespace {

constexpr int LANES = 16, V = 4;   // lanes over channels, channels per lane
constexpr int CT = LANES * V;      // channels of a tile
constexpr int ROW = CT + 4;        // floats a warp's row takes: no bank conflicts in join

// A CTA's shape: TEAMS teams of SCAN_TILE / L groups of LANES threads, a tile
// a team, L tokens a thread; and the warps that feed them.
template <int TOKENS> struct Shape {
    static constexpr int L = TOKENS, THREADS = SCAN_TILE / TOKENS * LANES, WARPS = THREADS / 32;
    static constexpr int TEAMS = 512 / THREADS;
    static constexpr int PARTS = THREADS / CT;     // threads per channel in join
    static_assert(WARPS == 2 * PARTS && 2 * L <= 32, "shape");
};
// A tile costs a thread some 400 instructions whatever its tokens, so the
// forward takes 16 a thread; the backward needs twice the registers a token.
using Fwd = Shape<16>;
using Bwd = Shape<8>;
constexpr int FEEDERS = 128, CTA = 512 + FEEDERS;
constexpr int RING = 196608;                       // bytes of all stages

constexpr int MAX_SEGMENTS = 256, MAX_UNITS = 1024;   // units: where there are segments
constexpr unsigned long long WAIT_NS = 2000000000ull;
constexpr unsigned ALL = 0xffffffffu;

// LA_ERR_TIMEOUT when a wait for a stage ran out (la_get_device_error).
__device__ int g_scan_error;

// ---- arithmetic -------------------------------------------------------------
// The kernels are as near to the issue rate as to HBM, so the channels go
// through the packed fp32 instructions two at a time.

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// exp(g).  Near 0 the decay is 1 + expm1(g) by its Taylor series (the next
// term, g^7 / 5040, is below 2^-26 of 1 for |g| < 1/4): the last addition is
// the only rounding of the size of the result, and it has no preferred sign.
// The hardware's 2^x has one (as has expf), and a channel that remembers
// thousands of tokens adds it up once a token: 1.1e-5 of the final state at
// 8192 tokens against 2e-6.  Elsewhere it is 2^x, which is within 2^-22, of
// g log2(e) rounded twice, the constant and the product: together within
// (4 + 1.25 |g|) 2^-24 of exp(g).  Gates below -1/4 forget within four tokens,
// so little of that adds up; gates above 1/4 do add it up while the state grows.
__device__ __forceinline__ F2 decay(F2 g)
{
    F2 p = fma2(g, f2(1.f / 720.f), f2(1.f / 120.f));
    p = fma2(g, p, f2(1.f / 24.f));
    p = fma2(g, p, f2(1.f / 6.f));
    p = fma2(g, p, f2(0.5f));
    p = fma2(mul2(g, g), p, g);
    const float2 near = un(add2(p, f2(1.f))), x = un(g), y = un(mul2(g, f2(1.44269504f)));
    return f2(fabsf(x.x) < 0.25f ? near.x : ex2(y.x), fabsf(x.y) < 0.25f ? near.y : ex2(y.y));
}

template <typename T> __device__ __forceinline__ float ldt(const T *p);
template <> __device__ __forceinline__ float ldt<float>(const float *p) { return *p; }
template <> __device__ __forceinline__ float ldt<__nv_bfloat16>(const __nv_bfloat16 *p)
{
    return __bfloat162float(*p);
}
template <typename T> __device__ __forceinline__ void stt(T *p, float x);
template <> __device__ __forceinline__ void stt<float>(float *p, float x) { *p = x; }
template <> __device__ __forceinline__ void stt<__nv_bfloat16>(__nv_bfloat16 *p, float x)
{
    *p = __float2bfloat16_rn(x);
}

// The values at a thread's V channels.
struct Val {
    F2 a, b;
    __device__ float4 f() const
    {
        const float2 x = un(a), y = un(b);
        return make_float4(x.x, x.y, y.x, y.y);
    }
};
__device__ __forceinline__ Val val(float a, float b, float c, float d)
{
    return Val{f2(a, b), f2(c, d)};
}
__device__ __forceinline__ Val val(float4 x) { return val(x.x, x.y, x.z, x.w); }
__device__ __forceinline__ Val fma2(const Val &x, const Val &y, const Val &z)
{
    return Val{fma2(x.a, y.a, z.a), fma2(x.b, y.b, z.b)};
}
__device__ __forceinline__ Val mul2(const Val &x, const Val &y)
{
    return Val{mul2(x.a, y.a), mul2(x.b, y.b)};
}
__device__ __forceinline__ Val add2(const Val &x, const Val &y)
{
    return Val{add2(x.a, y.a), add2(x.b, y.b)};
}
__device__ __forceinline__ Val decay(const Val &g) { return Val{decay(g.a), decay(g.b)}; }
__device__ __forceinline__ Val shuffled(const Val &x)   // from the warp's other group
{
    const float4 f = x.f();
    return val(__shfl_xor_sync(ALL, f.x, LANES), __shfl_xor_sync(ALL, f.y, LANES),
               __shfl_xor_sync(ALL, f.z, LANES), __shfl_xor_sync(ALL, f.w, LANES));
}

// As loaded: 8 bytes of bf16, 16 of fp32.
template <typename T> struct Four;
template <> struct Four<float> {
    float4 r;
    __device__ Val get() const { return val(r); }
    __device__ void set(const Val &v) { r = v.f(); }
};
template <> struct Four<__nv_bfloat16> {
    uint2 r;
    __device__ Val get() const
    {
        return val(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                   __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
    }
    __device__ void set(const Val &v)
    {
        const float4 f = v.f();
        const __nv_bfloat162 a = __floats2bfloat162_rn(f.x, f.y);
        const __nv_bfloat162 b = __floats2bfloat162_rn(f.z, f.w);
        r.x = *reinterpret_cast<const unsigned *>(&a);
        r.y = *reinterpret_cast<const unsigned *>(&b);
    }
};

// A product of decays that are not zero stays above zero where fp32 underflows:
// an infinite state stays infinite, as it does token by token (0 times infinity
// is NaN).  To a finite state the least fp32 number instead of 0 is as good: the
// underflow's own rounding.  b4 h32 d128 n8192 forward and backward: 371 us, 368
// without; 393 and 369 where every product of a thread underflows.
constexpr float LEAST = 1.4e-45f;   // 2^-149
__device__ __forceinline__ float times(float a, float b)
{
    const float r = a * b;
    return r == 0.f && a != 0.f && b != 0.f ? LEAST : r;
}
__device__ __forceinline__ bool some_zero(const Val &x)
{
    const float4 f = x.f();
    return fminf(fminf(f.x, f.y), fminf(f.z, f.w)) == 0.f;
}
__device__ __forceinline__ Val times(const Val &x, const Val &y)
{
    const Val r = mul2(x, y);
    if (!some_zero(r))
        return r;
    const float4 a = x.f(), b = y.f();
    return val(times(a.x, b.x), times(a.y, b.y), times(a.z, b.z), times(a.w, b.w));
}
// The same for A, the product of decays of which `least` are the smallest.
__device__ __forceinline__ Val above_zero(const Val &A, float4 least)
{
    auto at = [](float a, float l) { return a == 0.f && l != 0.f ? LEAST : a; };
    const float4 a = A.f();
    return val(at(a.x, least.x), at(a.y, least.y), at(a.z, least.z), at(a.w, least.w));
}
__device__ __forceinline__ void lower(float4 *least, const Val &d)
{
    const float4 f = d.f();
    *least = make_float4(fminf(least->x, f.x), fminf(least->y, f.y), fminf(least->z, f.z),
                         fminf(least->w, f.w));
}

// ---- tokens and channels -------------------------------------------------------

// The channels of a thread: V consecutive ones (VEC: one wide access each), or
// every LANES-th (any alignment).
template <bool VEC> __device__ __forceinline__ int local_channel(int lane, int v)
{
    return VEC ? lane * V + v : v * LANES + lane;
}

// The thread's part of a row of CT floats in shared memory.
template <bool VEC> __device__ __forceinline__ Val get_row(const float *row, int lane)
{
    if constexpr (VEC)
        return val(*reinterpret_cast<const float4 *>(row + lane * V));
    return val(row[lane], row[LANES + lane], row[2 * LANES + lane], row[3 * LANES + lane]);
}
template <bool VEC> __device__ __forceinline__ void put_row(float *row, int lane, const Val &v)
{
    const float4 f = v.f();
    if constexpr (VEC) {
        *reinterpret_cast<float4 *>(row + lane * V) = f;
    } else {
        row[lane] = f.x;
        row[LANES + lane] = f.y;
        row[2 * LANES + lane] = f.z;
        row[3 * LANES + lane] = f.w;
    }
}

// Which of a thread's channels are there.
template <bool VEC>
__device__ __forceinline__ unsigned present(unsigned c0, int lane, unsigned C)
{
    unsigned on = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
        on |= (c0 + local_channel<VEC>(lane, v) < C ? 1u : 0u) << v;
    return on;
}

// One token tensor as a thread sees it: its channels in a token's row.
template <typename T, bool VEC> struct Col {
    T *q;
    int64_t off[VEC ? 1 : V];
    // flat: the heads are D apart, so a channel's offset is its number
    __device__ Col(const void *base, int64_t sh, unsigned D, bool flat, unsigned c0, int lane,
                   unsigned on)
        : q(const_cast<T *>(static_cast<const T *>(base)))
    {
#pragma unroll
        for (int v = 0; v < (VEC ? 1 : V); ++v) {
            unsigned c = c0 + local_channel<VEC>(lane, v);
            c = on >> v & 1 ? c : 0;
            const int64_t o = flat ? c : c / D * sh + c % D;
            if constexpr (VEC)
                q += o;
            else
                off[v] = o;
        }
    }
    // four consecutive channels from c0 on
    __device__ Col(const void *base, int64_t sh, unsigned D, bool flat, unsigned c0, unsigned on)
        : q(const_cast<T *>(static_cast<const T *>(base)))
    {
#pragma unroll
        for (int v = 0; v < (VEC ? 1 : V); ++v) {
            const unsigned c = on >> v & 1 ? c0 + v : c0;   // (the others are not accessed)
            const int64_t o = flat ? c : c / D * sh + c % D;
            if constexpr (VEC)
                q += o;
            else
                off[v] = o;
        }
    }
    __device__ Four<T> four(const T *r, unsigned on) const
    {
        Four<T> x;
        if constexpr (VEC)
            x.r = *reinterpret_cast<const decltype(x.r) *>(r);
        else
            x.set(load(r, on));
        return x;
    }
    __device__ T *row(int b, int t, int64_t sb, int64_t st) const { return q + b * sb + t * st; }
    // one channel after the other, of rows that are not wide
    __device__ Val load(const T *r, unsigned on) const
    {
        float f[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            f[v] = on >> v & 1 ? ldt(r + off[VEC ? 0 : v]) : 0.f;
        return val(f[0], f[1], f[2], f[3]);
    }
    __device__ void store(T *r, unsigned on, const Val &x) const
    {
        if constexpr (VEC) {
            Four<T> w;
            w.set(x);
            *reinterpret_cast<decltype(w.r) *>(r) = w.r;
        } else {
            const float4 f = x.f();
            if (on & 1)
                stt(r + off[0], f.x);
            if (on & 2)
                stt(r + off[1], f.y);
            if (on & 4)
                stt(r + off[2], f.z);
            if (on & 8)
                stt(r + off[3], f.w);
        }
    }
};

// A state vector's values at four consecutive channels (0 where absent).
__device__ __forceinline__ Val get_state(const float *from, int64_t n, int64_t C, unsigned c0,
                                         unsigned on)
{
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        s[v] = from && (on >> v & 1) ? from[n * C + c0 + v] : 0.f;
    return val(s[0], s[1], s[2], s[3]);
}
__device__ __forceinline__ void put_state(float *to, int64_t n, int64_t C, unsigned c0,
                                          unsigned on, const Val &x)
{
    const float4 f = x.f();
    const float s[V] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (on >> v & 1)
            to[n * C + c0 + v] = s[v];
}

// The barrier of a team.
template <int N> struct Team {
    int id;   // 1 ..
    __device__ void sync() const { asm volatile("bar.sync %0, %1;" ::"r"(id), "n"(N) : "memory"); }
    __device__ bool all(bool x) const
    {
        unsigned r;
        asm volatile("{\n\t.reg .pred p, q;\n\t"
                     "setp.ne.u32 p, %1, 0;\n\t"
                     "bar.red.and.pred q, %2, %3, p;\n\t"
                     "selp.u32 %0, 1, 0, q;\n\t}"
                     : "=r"(r)
                     : "r"((unsigned)x), "r"(id), "n"(N)
                     : "memory");
        return r != 0;
    }
};

// ---- what a call is cut into ------------------------------------------------

struct Plan {
    int parts;          // of the channels
    int segments;       // of a sequence, in the order of the chain
    int units;          // sequences * segments * parts: what a team takes
    float2 *maps;       // [sequence][segment][C]: (A, B); A < 0: the state B itself
    int map;            // this launch forms them
    int group;          // GROUPED: teams that take a unit's tiles in turn (each a unit of its
                        // own); else 1
    int flat;           // every tensor's heads are D apart
    int small;          // no token stride is beyond 2^24
    int boxed;          // the tensors have their Boxes
    int withhold;       // diagnostic: the first tile of a CTA is not handed over
};

__device__ __forceinline__ unsigned long long now_ns()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// A sequence: its batch row, first token and tokens, and the first of its blocks
// of SIZE tokens among all sequences' (ScanArgs::states).
struct Row {
    int b, bos, len;
    int64_t block;
};
// ceil(n / SIZE), at every n
template <int SIZE> __device__ __forceinline__ int blocks_of(int n)
{
    return n / SIZE + (n % SIZE != 0);
}
template <int SIZE> __device__ __forceinline__ Row row_of(const ScanArgs &a, int n)
{
    if (!a.cu)
        return Row{n, 0, a.T, (int64_t)n * blocks_of<SIZE>(a.T)};
    // (within the tokens, whatever the table says by now)
    const int lo = min(max(a.cu[n], 0), a.T), hi = min(max(a.cu[n + 1], lo), a.T);
    return Row{0, lo, hi - lo, (int64_t)lo / SIZE + n};
}

// What a team needs to know of a tile.
struct Item {
    int stage;              // its place in the ring; < 0: no more
    int count;              // its tokens
    unsigned c0;            // its first channel
    int seq, segment;
    int begin, end;         // it is its unit's first, last
    int first, last;        // it holds its sequence's first, last token
    int b, t;               // of its first processed token
    int64_t block;          // its place in ScanArgs::states
};

template <class S, bool BACK> struct Maps {
    float A[S::WARPS][ROW], B[S::WARPS][ROW];   // the warps' maps
    float S_[S::WARPS][ROW];                    // the state that enters the warp
    // the backward's forward chain: B of the maps (A is the same), states
    float fB[BACK ? S::WARPS : 1][ROW], fS[BACK ? S::WARPS : 1][ROW];
};
template <class S, bool BACK, int NS> struct Shared {
    Maps<S, BACK> maps[S::TEAMS];
    Item item[S::TEAMS][2];       // a team's, in turn
    // at most two items of a team are under way: the feeding warps hand over the
    // next when one of the two barriers says that the last but one was worked off
    uint64_t full[S::TEAMS][2], done[S::TEAMS][2];
    uint64_t empty[NS];
    // of a group: the state after a tile, for the next one's team (a place for each
    // team: the tile that had the place before is then done)
    uint64_t passed[S::TEAMS / 2][S::TEAMS];
    float state[S::TEAMS / 2][S::TEAMS][CT];
    Item taken[2][S::TEAMS];      // by the feeders, in turn
};

// A group's way through its units: one lane's state.
struct Walk {
    int unit, step;     // the next unit; units apart
    int seq, seg, run;  // the present one
    int lo, jj, end;    // its tiles in the chain's order: [lo, end), jj done or next
    unsigned c0;
    Row row;
};
__device__ __forceinline__ bool enter_unit(const ScanArgs &a, const Plan &k, Walk *w)
{
    for (; w->unit < k.units; w->unit += w->step) {
        const int u = w->unit / k.parts;
        w->c0 = (unsigned)(w->unit - u * k.parts) * CT;
        w->seq = u / k.segments;
        w->seg = u - w->seq * k.segments;
        w->row = row_of<SCAN_TILE>(a, w->seq);
        w->run = blocks_of<SCAN_TILE>(w->row.len);
        const int len = (w->run + k.segments - 1) / k.segments;
        w->lo = w->jj = w->seg * len;
        w->end = min(w->jj + len, w->run);
        // (of the last segment nobody needs the map)
        if (w->jj >= w->end || (k.map && w->end == w->run))
            continue;
        w->unit += w->step;
        return true;
    }
    w->jj = w->end = 0;
    return false;
}

template <bool BACK>
__device__ __forceinline__ Item next_item(const ScanArgs &a, const Plan &k, Walk *w)
{
    Item d;
    d.stage = -1;
    d.begin = 0;
    if (w->jj >= w->end) {
        if (!enter_unit(a, k, w))
            return d;
        d.begin = 1;
    }
    d.stage = 0;
    // the first pass goes through a segment backwards: what it reads last, the
    // second pass reads first, while L2 still has it
    const int jj = k.map ? w->lo + w->end - 1 - w->jj : w->jj;
    const int j = BACK ? w->run - 1 - jj : jj, p = j * SCAN_TILE;
    d.count = min(w->row.len - p, SCAN_TILE);
    d.c0 = w->c0;
    d.seq = w->seq;
    d.segment = w->seg;
    d.end = ++w->jj == w->end;
    d.first = j == 0;
    d.last = j == w->run - 1;
    d.b = w->row.b;
    d.t = w->row.bos + (a.reverse ? w->row.len - 1 - p : p);
    d.block = w->row.block + j;
    return d;
}

// What PARTS neighbouring lanes know of a channel's maps: part p holds those of
// the warps 2p and 2p + 1 in the order of the chain (BACK: the last warp first).
struct Run {
    float A0, B0;   // the first warp's map
    float eA, eB;   // the map of all warps before it
    float A, B;     // the map of the tile (in every lane)
};
template <class S, bool BACK>
__device__ __forceinline__ Run run_of(const float (&A)[S::WARPS][ROW],
                                      const float (&B)[S::WARPS][ROW])
{
    constexpr int PARTS = S::PARTS;
    const int c = threadIdx.x % S::THREADS / PARTS, part = threadIdx.x % PARTS;
    const int w0 = BACK ? S::WARPS - 1 - 2 * part : 2 * part, w1 = BACK ? w0 - 1 : w0 + 1;
    Run q;
    q.A0 = A[w0][c];
    q.B0 = B[w0][c];
    q.A = times(q.A0, A[w1][c]);
    q.B = fmaf(A[w1][c], q.B0, B[w1][c]);
#pragma unroll
    for (int i = 1; i < PARTS; i *= 2) {
        const float x = __shfl_up_sync(ALL, q.A, i), y = __shfl_up_sync(ALL, q.B, i);
        if (part >= i) {
            q.B = fmaf(q.A, y, q.B);
            q.A = times(q.A, x);
        }
    }
    q.eA = __shfl_up_sync(ALL, q.A, 1);
    q.eB = __shfl_up_sync(ALL, q.B, 1);
    if (part == 0)
        q.eA = 1.f, q.eB = 0.f;
    const int last = threadIdx.x % 32 / PARTS * PARTS + PARTS - 1;
    q.A = __shfl_sync(ALL, q.A, last);
    q.B = __shfl_sync(ALL, q.B, last);
    return q;
}
// The states that enter the warps, from the one that enters the tile.
template <class S, bool BACK>
__device__ __forceinline__ void spread(float (&to)[S::WARPS][ROW], const Run &q, float s)
{
    const int c = threadIdx.x % S::THREADS / S::PARTS, part = threadIdx.x % S::PARTS;
    const int w0 = BACK ? S::WARPS - 1 - 2 * part : 2 * part, w1 = BACK ? w0 - 1 : w0 + 1;
    const float in = fmaf(q.eA, s, q.eB);
    to[w0][c] = in;
    to[w1][c] = fmaf(q.A0, in, q.B0);
}

// What the PARTS lanes of a channel carry from tile to tile: the state, or in the
// first pass the map (A, s) of the tiles from here to the segment's end.
struct Carry {
    float s, A;
};
// The unit's first tile: what it starts from; init: the sequence's.
__device__ __forceinline__ void start(const Plan &k, const Item &it, const float *init, int64_t C,
                                      int64_t c, Carry *x)
{
    x->s = 0.f;
    x->A = 1.f;
    if (k.map || c >= C)
        return;
    if (it.segment == 0) {
        if (init)
            x->s = init[it.seq * C + c];
        return;
    }
    const float2 *m = k.maps + (int64_t)it.seq * k.segments * C + c;
    constexpr int BATCH = 8;
    for (int i = 0; i < it.segment; i += BATCH) {
        float2 v[BATCH];
#pragma unroll
        for (int u = 0; u < BATCH; ++u)
            v[u] = i + u < it.segment ? m[(i + u) * C] : make_float2(1.f, 0.f);
#pragma unroll
        for (int u = 0; u < BATCH; ++u)
            x->s = v[u].x < 0.f ? v[u].y : fmaf(v[u].x, x->s, v[u].y);
    }
}
// The tile's map is known: hands the state that enters it to the warps and steps
// over the tile; after the chain's last tile its state.  First pass: takes the
// tile in front of the map, which it writes after the segment's last tile (for a
// sequence's first segment the state at its end).
template <class S, bool BACK>
__device__ __forceinline__ void step(const Plan &k, const Item &it, Maps<S, BACK> &maps, int64_t C,
                                     int64_t c, const float *init, float *fin, Carry *x)
{
    const Run q = run_of<S, BACK>(maps.A, maps.B);
    const bool speaks = threadIdx.x % S::PARTS == 0 && c < C;
    if (k.map) {
        x->s = fmaf(x->A, q.B, x->s);
        x->A = times(x->A, q.A);
        if (it.end && speaks) {
            float2 m = make_float2(x->A, x->s);
            if (it.segment == 0)
                m = make_float2(-1.f, init ? fmaf(x->A, init[it.seq * C + c], x->s) : x->s);
            k.maps[((int64_t)it.seq * k.segments + it.segment) * C + c] = m;
        }
        return;
    }
    spread<S, BACK>(maps.S_, q, x->s);
    x->s = fmaf(q.A, x->s, q.B);
    if ((BACK ? it.first : it.last) && fin && speaks)
        fin[it.seq * C + c] = x->s;
}

// ---- the ring ---------------------------------------------------------------
// A stage holds [SCAN_TILE][CT] of x, then of g, then (BACK) of do, by position.

template <bool BACK, typename T, typename TG> struct Stage {
    static constexpr int X = SCAN_TILE * CT * (int)sizeof(T), G = SCAN_TILE * CT * (int)sizeof(TG);
    static constexpr int BYTES = X * (BACK ? 2 : 1) + G, NS = RING / BYTES;
};

// mbarrier waits: at most WAIT_NS, then the error word.  false: it ran out.
__device__ __forceinline__ bool stage_wait(uint64_t *bar, unsigned parity)
{
    if (sm100::mbar_try_wait(bar, parity))
        return true;
    const unsigned long long t0 = now_ns();
    while (!sm100::mbar_try_wait(bar, parity)) {
        if (now_ns() - t0 > WAIT_NS) {
            atomicExch(&g_scan_error, LA_ERR_TIMEOUT);
            return false;
        }
    }
    return true;
}

// The group's tile number m: takes the state over from the team of the tile
// before it.  A unit's first tile (begin) has its own state to start from and
// only waits, so that the places keep their order.
template <class S, bool BACK, int NS>
__device__ __forceinline__ bool taken_over(Shared<S, BACK, NS> &sm, int group, unsigned m,
                                           int begin, Carry *x)
{
    if (m == 0)
        return true;
    --m;
    if (!stage_wait(&sm.passed[group][m % S::TEAMS], m / S::TEAMS & 1))
        return false;
    if (!begin)
        x->s = sm.state[group][m % S::TEAMS][threadIdx.x % S::THREADS / S::PARTS];
    return true;
}
template <class S, bool BACK, int NS>
__device__ __forceinline__ void pass_on(Shared<S, BACK, NS> &sm, int group, unsigned m,
                                        const Carry &x)
{
    if (threadIdx.x % S::PARTS == 0)
        sm.state[group][m % S::TEAMS][threadIdx.x % S::THREADS / S::PARTS] = x.s;
    sm100::mbar_arrive(&sm.passed[group][m % S::TEAMS]);
}

// Bytes from a token's row to the next processed token's (Plan::small).
template <typename T> __device__ __forceinline__ int step_of(const ScanArgs &a, int64_t st)
{
    const int b = (int)st * (int)sizeof(T);
    return a.reverse ? -b : b;
}
template <typename T> __device__ __forceinline__ T *stepped(T *r, int e, int step)
{
    return reinterpret_cast<T *>(reinterpret_cast<intptr_t>(r) + (int64_t)e * step);
}

__device__ __forceinline__ void expect(uint64_t *bar, unsigned bytes)
{
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(
                     sm100::smem_u32(bar)),
                 "r"(bytes)
                 : "memory");
}

// A feeding lane copies token i's row of the tile, of one tensor: one copy, or
// one for each head where the heads are apart.
template <typename T>
__device__ __forceinline__ void copy_row(const ScanArgs &a, const Tok &x, const Item &it, int t,
                                         bool flat, unsigned C, int row, uint8_t *to,
                                         uint64_t *full)
{
    const T *q = static_cast<const T *>(x.p) + it.b * x.sb + t * x.st;
    const unsigned end = min(it.c0 + CT, C);
    uint32_t dst = sm100::smem_u32(to) + row * CT * (unsigned)sizeof(T);
    for (unsigned c = it.c0; c < end;) {
        const unsigned h = flat ? 0 : c / a.D, d = flat ? c : c - h * a.D;
        const unsigned n = flat ? end - c : min(end - c, a.D - d);
        asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1], %2, [%3];" ::"r"(dst),
                     "l"(q + h * x.sh + d), "r"(n * (unsigned)sizeof(T)),
                     "r"(sm100::smem_u32(full))
                     : "memory");
        dst += n * (unsigned)sizeof(T);
        c += n;
    }
}

// Boxes of SCAN_TILE tokens and CT channels {channel, head, token, batch row}.
struct Boxes {
    CUtensorMap x, g, d;
};

// The feeding warps: FLIP (reverse): the tile's last token is its first row.
template <class S, bool BACK, typename T, typename TG, bool VEC, bool FLIP>
__device__ __forceinline__ void feed(const ScanArgs &a, const Plan &k, const Boxes &boxes,
                                     Shared<S, BACK, Stage<BACK, T, TG>::NS> &sm, uint8_t *ring,
                                     unsigned C)
{
    using St = Stage<BACK, T, TG>;
    const Team<FEEDERS> team{15};
    const int lane = threadIdx.x % 32, w = (threadIdx.x - 512) / 32;
    const bool needs_x = !BACK || !k.map;
    const int groups = S::TEAMS / k.group;
    Walk walk{};   // of group `lane`
    walk.unit = blockIdx.x + lane * gridDim.x;
    walk.step = gridDim.x * groups;
    unsigned q = 0;              // stages handed out
    unsigned ended = 0;          // bit i: team i has been told so
    for (unsigned n = 0; ended != (1u << S::TEAMS) - 1; ++n) {   // every team's n-th tile
        if (w == 0 && lane < groups)
            for (int i = 0; i < k.group; ++i)
                sm.taken[n & 1][lane * k.group + i] = next_item<BACK>(a, k, &walk);
        team.sync();
        for (int i = 0; i < S::TEAMS; ++i) {
            if (ended >> i & 1)
                continue;
            const Item &it = sm.taken[n & 1][i];
            const bool none = it.stage < 0;
            const unsigned st = q % St::NS, used = q / St::NS;
            bool ok = n < 2 || stage_wait(&sm.done[i][n & 1], (n / 2 - 1) & 1);
            if (!none)
                ok = (!used || stage_wait(&sm.empty[st], (used - 1) & 1)) && ok;
            if (!team.all(ok))
                return;
            uint64_t *full = &sm.full[i][n & 1];
            if (w == 0 && lane == 0) {
                sm.item[i][n & 1] = it;
                if (!none)
                    sm.item[i][n & 1].stage = (int)st;
            }
            if (none) {
                ended |= 1u << i;
            } else {
                ++q;
                uint8_t *to = ring + st * St::BYTES;
                const int t = threadIdx.x - 512;   // the lane's token
                // the bytes are announced first: they may land before the arrival
                if (VEC && k.boxed) {
                    if (t == 0) {
                        const int h = k.flat ? 0 : it.c0 / a.D, c = it.c0 - h * a.D;
                        const int t0 = FLIP ? it.t - (SCAN_TILE - 1) : it.t;
                        expect(full, St::BYTES - (needs_x ? 0 : St::X));
                        if (needs_x)
                            sm100::tma_load_4d(to, &boxes.x, full, c, h, t0, it.b);
                        sm100::tma_load_4d(to + St::X, &boxes.g, full, c, h, t0, it.b);
                        if (BACK)
                            sm100::tma_load_4d(to + St::X + St::G, &boxes.d, full, c, h, t0, it.b);
                    }
                } else if (VEC && t < it.count) {
                    const int row = FLIP ? SCAN_TILE - 1 - t : t, at = it.t + (FLIP ? -t : t);
                    const int per = (int)(sizeof(TG) + (needs_x ? sizeof(T) : 0) +
                                          (BACK ? sizeof(T) : 0));
                    expect(full, (min(it.c0 + CT, C) - it.c0) * per);
                    if (needs_x)
                        copy_row<T>(a, a.x, it, at, k.flat, C, row, to, full);
                    copy_row<TG>(a, a.g, it, at, k.flat, C, row, to + St::X, full);
                    if (BACK)
                        copy_row<T>(a, a.d_o, it, at, k.flat, C, row, to + St::X + St::G, full);
                }
            }
            if (!(k.withhold && n == 0 && i == 0))
                sm100::mbar_arrive(full);
        }
    }
    // copies under way end before the CTA does: every one is waited for by the
    // team that it is for, unless a wait ran out, long after they have landed
}

// The thread's values in a stage: token e of the group at [e * pitch].
template <typename T, bool FLIP>
__device__ __forceinline__ Four<T> *values(uint8_t *tile, int lane, int slot)
{
    return reinterpret_cast<Four<T> *>(tile) + (FLIP ? SCAN_TILE - 1 - slot : slot) * (CT / V) +
           lane;
}

// Rows that no wide access fits: the team itself loads them, eight tokens of a
// thread at a time.  Without conditions (absent channels and tokens are read from
// another's place), so that the loads are under way together.
template <int PITCH, typename T>
__device__ __forceinline__ void fill(Four<T> *to, const Col<T, false> &c, const T *row, int64_t by,
                                     int count)
{
    constexpr int AT = 8;
#pragma unroll 1
    for (int e0 = 0; e0 < count; e0 += AT) {
        T v[AT][V];
#pragma unroll
        for (int e = 0; e < AT; ++e) {
            const T *r = row + min(e0 + e, count - 1) * by;
#pragma unroll
            for (int u = 0; u < V; ++u)
                v[e][u] = r[c.off[u]];
        }
#pragma unroll
        for (int e = 0; e < AT; ++e)
            if (e0 + e < count)
                to[(e0 + e) * PITCH].set(val(ldt(&v[e][0]), ldt(&v[e][1]), ldt(&v[e][2]),
                                             ldt(&v[e][3])));
    }
}

template <class S, bool BACK, int NS>
__device__ __forceinline__ void set_up(Shared<S, BACK, NS> &sm)
{
    if (threadIdx.x == 0) {
        for (int i = 0; i < S::TEAMS; ++i) {
            for (int u = 0; u < 2; ++u) {
                sm100::mbar_init(&sm.full[i][u], FEEDERS);
                sm100::mbar_init(&sm.done[i][u], S::THREADS);
            }
            for (int u = 0; u < S::TEAMS / 2; ++u)
                sm100::mbar_init(&sm.passed[u][i], S::THREADS);
        }
        for (int i = 0; i < NS; ++i)
            sm100::mbar_init(&sm.empty[i], S::THREADS);
        sm100::fence_mbar_init();
    }
    __syncthreads();
}

// 96 registers a thread at the launch: 640 x 96 = 512 x 104 + 128 x 64.
__device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;" ::: "memory");
}
__device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;" ::: "memory");
}

// ---- forward ----------------------------------------------------------------

template <typename T, typename TG, bool VEC, bool FLIP, bool GROUPED>
__global__ void __launch_bounds__(CTA, 1)
    scan_fwd_tiles(const ScanArgs a, const Plan k, const __grid_constant__ Boxes boxes)
{
    using S = Fwd;
    using St = Stage<false, T, TG>;
    constexpr int L = S::L, PARTS = S::PARTS, PITCH = FLIP ? -CT / V : CT / V;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Shared<S, false, St::NS> sm;
    const unsigned C = (unsigned)a.H * (unsigned)a.D;
    set_up(sm);
    if (threadIdx.x >= 512) {
        fewer_registers();
        feed<S, false, T, TG, VEC, FLIP>(a, k, boxes, sm, ring, C);
        return;
    }
    more_registers();
    const int me = threadIdx.x % S::THREADS, lane = me % LANES, slot = me / LANES * L;
    const int warp = me / 32, dir = a.reverse ? -1 : 1;
    const bool odd = me & LANES;   // the second group of the warp
    const Team<S::THREADS> team{1 + (int)threadIdx.x / S::THREADS};
    Maps<S, false> &maps = sm.maps[team.id - 1];
    const int group = (team.id - 1) / k.group, place = (team.id - 1) % k.group;
    Carry carry{0.f, 1.f};
    for (unsigned n = 0;; ++n) {
        if (!team.all(stage_wait(&sm.full[team.id - 1][n & 1], n / 2 & 1)))
            break;
        const Item &it = sm.item[team.id - 1][n & 1];
        const int st = it.stage;
        if (st < 0)
            break;
        const unsigned c0 = it.c0, ch = c0 + me / PARTS;   // ch: the channel of step
        if (it.begin)
            start(k, it, a.init, C, ch, &carry);
        uint8_t *tile = ring + st * St::BYTES;
        Four<T> *xs = values<T, FLIP>(tile, lane, slot);
        Four<TG> *gs = values<TG, FLIP>(tile + St::X, lane, slot);
        const unsigned on = present<VEC>(c0, lane, C);
        const int count = on ? max(0, min(L, it.count - slot)) : 0;
        const bool plain = k.small && count == L;
        const int b = it.b, t0 = it.t + dir * slot;   // the group's first token
        if constexpr (!VEC) {
            const Col<T, VEC> x(a.x.p, a.x.sh, a.D, k.flat, c0, lane, on);
            const Col<TG, VEC> g(a.g.p, a.g.sh, a.D, k.flat, c0, lane, on);
            fill<PITCH>(xs, x, x.row(b, t0, a.x.sb, a.x.st), dir * a.x.st, count);
            fill<PITCH>(gs, g, g.row(b, t0, a.g.sb, a.g.st), dir * a.g.st, count);
        }
        // the thread's tokens composed to s -> A s + B.  Their decays are kept
        // for the second pass, in the stage: the registers for them would cost
        // warps.  fp32 gates are replaced by theirs; a bf16 gate and its x
        // together have the decay's size, and x goes to registers meanwhile.
        constexpr bool KEEP = sizeof(TG) == 2;
        Four<T> keep[KEEP ? L : 1];
        Val A = val(1.f, 1.f, 1.f, 1.f), B = val(0.f, 0.f, 0.f, 0.f);
        if (plain) {
#pragma unroll
            for (int e = 0; e < L; ++e) {
                const Val d = decay(gs[e * PITCH].get());
                const Four<T> x = xs[e * PITCH];
                B = fma2(d, B, x.get());
                A = mul2(A, d);
                if constexpr (KEEP) {
                    keep[e] = x;
                    reinterpret_cast<unsigned long long *>(xs)[e * PITCH] = d.a.v;
                    reinterpret_cast<unsigned long long *>(gs)[e * PITCH] = d.b.v;
                } else {
                    gs[e * PITCH].set(d);
                }
            }
        } else {
#pragma unroll 1
            for (int e = 0; e < count; ++e) {
                const Val d = decay(gs[e * PITCH].get());
                B = fma2(d, B, xs[e * PITCH].get());
                A = mul2(A, d);
            }
        }
        if (some_zero(A)) {   // (gates of -6.5 and below on the average)
            float4 least = make_float4(1.f, 1.f, 1.f, 1.f);
#pragma unroll 1
            for (int e = 0; e < count; ++e) {
                if (!plain) {
                    lower(&least, decay(gs[e * PITCH].get()));
                } else if constexpr (KEEP) {
                    lower(&least, Val{{reinterpret_cast<unsigned long long *>(xs)[e * PITCH]},
                                      {reinterpret_cast<unsigned long long *>(gs)[e * PITCH]}});
                } else {
                    lower(&least, gs[e * PITCH].get());
                }
            }
            A = above_zero(A, least);
        }
        // the two groups of a warp, then the warps
        const Val eA = shuffled(A), eB = shuffled(B);   // the other group's map
        if (odd) {
            put_row<VEC>(maps.A[warp], lane, times(A, eA));
            put_row<VEC>(maps.B[warp], lane, fma2(A, eB, B));
        }
        if (GROUPED) {
            if (!team.all(taken_over(sm, group, n * k.group + place, it.begin,
                                     &carry)))
                break;
        } else {
            team.sync();
        }
        if (a.states && !it.first && !k.map && me % PARTS == 0 && ch < C)
            a.states[it.block * C + ch] = carry.s;
        step<S, false>(k, it, maps, C, ch, a.init, a.fin, &carry);
        if (GROUPED)
            pass_on(sm, group, n * k.group + place, carry);
        team.sync();
        if (count && !k.map && a.o.p) {
            Val s = get_row<VEC>(maps.S_[warp], lane);
            if (odd)
                s = fma2(eA, s, eB);
            const Col<T, VEC> o(a.o.p, a.o.sh, a.D, k.flat, c0, lane, on);
            if (plain) {
                T *const row = o.row(b, t0, a.o.sb, a.o.st);
                const int by = step_of<T>(a, a.o.st);
#pragma unroll
                for (int e = 0; e < L; ++e) {
                    if constexpr (KEEP)
                        s = fma2(Val{{reinterpret_cast<unsigned long long *>(xs)[e * PITCH]},
                                     {reinterpret_cast<unsigned long long *>(gs)[e * PITCH]}},
                                 s, keep[e].get());
                    else
                        s = fma2(gs[e * PITCH].get(), s, xs[e * PITCH].get());
                    o.store(stepped(row, e, by), on, s);
                }
            } else {
#pragma unroll 1
                for (int e = 0; e < count; ++e) {
                    s = fma2(decay(gs[e * PITCH].get()), s, xs[e * PITCH].get());
                    o.store(o.row(b, t0 + dir * e, a.o.sb, a.o.st), on, s);
                }
            }
        }
        sm100::fence_proxy_async_smem();   // this thread's writes there, before the next copy's
        sm100::mbar_arrive(&sm.empty[st]);
        sm100::mbar_arrive(&sm.done[team.id - 1][n & 1]);
    }
}

// ---- backward -----------------------------------------------------------------
// The chain runs from the last token to the first; s_{t-1} comes from the states
// that entered the tiles in the forward.

template <typename T, typename TG, bool VEC, bool FLIP, bool GROUPED>
__global__ void __launch_bounds__(CTA, 1)
    scan_bwd_tiles(const ScanArgs a, const Plan k, const __grid_constant__ Boxes boxes)
{
    using S = Bwd;
    using St = Stage<true, T, TG>;
    constexpr int L = S::L, PARTS = S::PARTS, PITCH = FLIP ? -CT / V : CT / V;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Shared<S, true, St::NS> sm;
    const unsigned C = (unsigned)a.H * (unsigned)a.D;
    set_up(sm);
    if (threadIdx.x >= 512) {
        fewer_registers();
        feed<S, true, T, TG, VEC, FLIP>(a, k, boxes, sm, ring, C);
        return;
    }
    more_registers();
    const int me = threadIdx.x % S::THREADS, lane = me % LANES, slot = me / LANES * L;
    const int warp = me / 32, dir = a.reverse ? -1 : 1;
    const bool odd = me & LANES;
    const Team<S::THREADS> team{1 + (int)threadIdx.x / S::THREADS};
    Maps<S, true> &maps = sm.maps[team.id - 1];
    const int group = (team.id - 1) / k.group, place = (team.id - 1) % k.group;
    Carry carry{0.f, 1.f};
    for (unsigned n = 0;; ++n) {
        if (!team.all(stage_wait(&sm.full[team.id - 1][n & 1], n / 2 & 1)))
            break;
        const Item &it = sm.item[team.id - 1][n & 1];
        const int st = it.stage;
        if (st < 0)
            break;
        const unsigned c0 = it.c0, ch = c0 + me / PARTS;   // ch: the channel of step
        if (it.begin)
            start(k, it, a.dfin, C, ch, &carry);
        uint8_t *tile = ring + st * St::BYTES;
        Four<T> *xs = values<T, FLIP>(tile, lane, slot);
        Four<TG> *gs = values<TG, FLIP>(tile + St::X, lane, slot);
        Four<T> *ds = values<T, FLIP>(tile + St::X + St::G, lane, slot);
        // the forward state that enters the tile
        float fs = 0.f;
        if (!k.map && ch < C) {
            if (!it.first)
                fs = a.states[it.block * C + ch];
            else if (a.init)
                fs = a.init[(int64_t)it.seq * C + ch];
        }
        const unsigned on = present<VEC>(c0, lane, C);
        const int count = on ? max(0, min(L, it.count - slot)) : 0;
        const bool plain = k.small && count == L;
        const int b = it.b, t0 = it.t + dir * slot;   // the group's first token
        if constexpr (!VEC) {
            const Col<T, VEC> xc(a.x.p, a.x.sh, a.D, k.flat, c0, lane, on);
            const Col<T, VEC> dc(a.d_o.p, a.d_o.sh, a.D, k.flat, c0, lane, on);
            const Col<TG, VEC> gc(a.g.p, a.g.sh, a.D, k.flat, c0, lane, on);
            fill<PITCH>(xs, xc, xc.row(b, t0, a.x.sb, a.x.st), dir * a.x.st, count);
            fill<PITCH>(gs, gc, gc.row(b, t0, a.g.sb, a.g.st), dir * a.g.st, count);
            fill<PITCH>(ds, dc, dc.row(b, t0, a.d_o.sb, a.d_o.st), dir * a.d_o.st, count);
        }
        // the thread's maps of the forward chain (A, fB) and of the backward
        // chain (A, B): the same decays, one product.  B from the first token
        // on: K = A K' + B with A = d_0 .. d_e, B = sum_i d_0 .. d_i do_i
        Val d[L], A = val(1.f, 1.f, 1.f, 1.f), B = val(0.f, 0.f, 0.f, 0.f), fB = B;
#pragma unroll
        for (int e = 0; e < L; ++e) {
            if (e < count) {
                d[e] = decay(gs[e * PITCH].get());
                fB = fma2(d[e], fB, xs[e * PITCH].get());
                A = mul2(A, d[e]);
                B = fma2(A, ds[e * PITCH].get(), B);
            }
        }
        if (some_zero(A)) {
            // B token by token then: 0 times an infinite do is not what the chain gives
            float4 least = make_float4(1.f, 1.f, 1.f, 1.f);
            B = val(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int e = L - 1; e >= 0; --e) {
                if (e < count) {
                    lower(&least, d[e]);
                    B = mul2(d[e], add2(ds[e * PITCH].get(), B));
                }
            }
            A = above_zero(A, least);
        }
        // the other group's maps: the even group's forward one for the odd, the
        // odd group's backward one for the even
        const Val oA = shuffled(A), oB = shuffled(odd ? B : fB);
        if (odd) {
            put_row<VEC>(maps.fB[warp], lane, fma2(A, oB, fB));
        } else {
            put_row<VEC>(maps.A[warp], lane, times(A, oA));
            put_row<VEC>(maps.B[warp], lane, fma2(A, oB, B));
        }
        if (GROUPED) {
            if (!team.all(taken_over(sm, group, n * k.group + place, it.begin,
                                     &carry)))
                break;
        } else {
            team.sync();
        }
        if (!k.map)
            spread<S, false>(maps.fS, run_of<S, false>(maps.A, maps.fB), fs);
        step<S, true>(k, it, maps, C, ch, a.dfin, a.dinit, &carry);
        if (GROUPED)
            pass_on(sm, group, n * k.group + place, carry);
        team.sync();
        if (count && !k.map) {
            Val s = get_row<VEC>(maps.fS[warp], lane), K = get_row<VEC>(maps.S_[warp], lane);
            if (odd)
                s = fma2(oA, s, oB);
            else
                K = fma2(oA, K, oB);
            const Col<T, VEC> dx(a.dx.p, a.dx.sh, a.D, k.flat, c0, lane, on);
            const Col<TG, VEC> dg(a.dg.p, a.dg.sh, a.D, k.flat, c0, lane, on);
            Val x[L];   // the states before the thread's tokens
#pragma unroll
            for (int e = 0; e < L; ++e) {
                if (e < count) {
                    x[e] = s;
                    s = fma2(d[e], s, xs[e * PITCH].get());
                }
            }
            T *const xr = dx.row(b, t0, a.dx.sb, a.dx.st);
            TG *const gr = dg.row(b, t0, a.dg.sb, a.dg.st);
            if (plain) {
                const int xd = step_of<T>(a, a.dx.st), gd = step_of<TG>(a, a.dg.st);
#pragma unroll
                for (int e = L - 1; e >= 0; --e) {
                    const Val G = add2(ds[e * PITCH].get(), K);
                    K = mul2(d[e], G);
                    dx.store(stepped(xr, e, xd), on, G);
                    dg.store(stepped(gr, e, gd), on, mul2(K, x[e]));
                }
            } else {
#pragma unroll
                for (int e = L - 1; e >= 0; --e) {
                    if (e < count) {
                        const Val G = add2(ds[e * PITCH].get(), K);
                        K = mul2(d[e], G);
                        dx.store(xr + dir * e * a.dx.st, on, G);
                        dg.store(gr + dir * e * a.dg.st, on, mul2(K, x[e]));
                    }
                }
            }
        }
        sm100::mbar_arrive(&sm.empty[st]);
        sm100::mbar_arrive(&sm.done[team.id - 1][n & 1]);
    }
}

// ---- serial ---------------------------------------------------------------------
// A thread takes four channels of a sequence and walks it alone, SCAN_BLOCK
// tokens at a time, whose loads are under way together.

template <typename T, typename TG, bool VEC>
__global__ void __launch_bounds__(128) scan_fwd_serial(const ScanArgs a, int flat)
{
    const unsigned C = (unsigned)a.H * (unsigned)a.D, quads = (C + V - 1) / V;
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (i >= (int64_t)a.N * quads)
        return;
    const int n = (int)(i / quads), dir = a.reverse ? -1 : 1;
    const unsigned c0 = (unsigned)(i - (int64_t)n * quads) * V;
    const Row w = row_of<SCAN_BLOCK>(a, n);
    const unsigned on = (1u << min(C - c0, (unsigned)V)) - 1;
    const Col<T, VEC> x(a.x.p, a.x.sh, a.D, flat, c0, on), o(a.o.p, a.o.sh, a.D, flat, c0, on);
    const Col<TG, VEC> g(a.g.p, a.g.sh, a.D, flat, c0, on);
    Val s = get_state(a.init, n, C, c0, on);
    const int t0 = w.bos + (a.reverse ? w.len - 1 : 0);
    for (int p = 0; p < w.len; p += SCAN_BLOCK) {
        Four<T> xr[SCAN_BLOCK];
        Four<TG> gr[SCAN_BLOCK];
#pragma unroll
        for (int e = 0; e < SCAN_BLOCK; ++e) {
            if (p + e < w.len) {
                const int t = t0 + dir * (p + e);
                xr[e] = x.four(x.row(w.b, t, a.x.sb, a.x.st), on);
                gr[e] = g.four(g.row(w.b, t, a.g.sb, a.g.st), on);
            }
        }
        if (a.states && p)
            put_state(a.states, w.block + p / SCAN_BLOCK, C, c0, on, s);
#pragma unroll
        for (int e = 0; e < SCAN_BLOCK; ++e) {
            if (p + e < w.len) {
                s = fma2(decay(gr[e].get()), s, xr[e].get());
                if (a.o.p)
                    o.store(o.row(w.b, t0 + dir * (p + e), a.o.sb, a.o.st), on, s);
            }
        }
    }
    if (a.fin)
        put_state(a.fin, n, C, c0, on, s);
}

template <typename T, typename TG, bool VEC>
__global__ void __launch_bounds__(128) scan_bwd_serial(const ScanArgs a, int flat)
{
    const unsigned C = (unsigned)a.H * (unsigned)a.D, quads = (C + V - 1) / V;
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (i >= (int64_t)a.N * quads)
        return;
    const int n = (int)(i / quads), dir = a.reverse ? -1 : 1;
    const unsigned c0 = (unsigned)(i - (int64_t)n * quads) * V;
    const Row w = row_of<SCAN_BLOCK>(a, n);
    const unsigned on = (1u << min(C - c0, (unsigned)V)) - 1;
    const Col<T, VEC> x(a.x.p, a.x.sh, a.D, flat, c0, on), d(a.d_o.p, a.d_o.sh, a.D, flat, c0, on);
    const Col<T, VEC> dx(a.dx.p, a.dx.sh, a.D, flat, c0, on);
    const Col<TG, VEC> g(a.g.p, a.g.sh, a.D, flat, c0, on), dg(a.dg.p, a.dg.sh, a.D, flat, c0, on);
    Val K = get_state(a.dfin, n, C, c0, on);
    const int t0 = w.bos + (a.reverse ? w.len - 1 : 0);
    for (int p = (w.len - 1) / SCAN_BLOCK * SCAN_BLOCK; p >= 0 && w.len > 0; p -= SCAN_BLOCK) {
        Val dec[SCAN_BLOCK], prev[SCAN_BLOCK], grad[SCAN_BLOCK];
#pragma unroll
        for (int e = 0; e < SCAN_BLOCK; ++e) {
            if (p + e < w.len) {
                const int t = t0 + dir * (p + e);
                prev[e] = x.four(x.row(w.b, t, a.x.sb, a.x.st), on).get();
                dec[e] = g.four(g.row(w.b, t, a.g.sb, a.g.st), on).get();
                grad[e] = d.four(d.row(w.b, t, a.d_o.sb, a.d_o.st), on).get();
            }
        }
        Val s = p ? get_state(a.states, w.block + p / SCAN_BLOCK, C, c0, on)
                  : get_state(a.init, n, C, c0, on);
#pragma unroll
        for (int e = 0; e < SCAN_BLOCK; ++e) {
            if (p + e < w.len) {
                dec[e] = decay(dec[e]);
                const Val y = fma2(dec[e], s, prev[e]);
                prev[e] = s;
                s = y;
            }
        }
#pragma unroll
        for (int e = SCAN_BLOCK - 1; e >= 0; --e) {
            if (p + e < w.len) {
                const int t = t0 + dir * (p + e);
                const Val G = add2(grad[e], K);
                K = mul2(dec[e], G);
                dx.store(dx.row(w.b, t, a.dx.sb, a.dx.st), on, G);
                dg.store(dg.row(w.b, t, a.dg.sb, a.dg.st), on, mul2(K, prev[e]));
            }
        }
    }
    if (a.dinit)
        put_state(a.dinit, n, C, c0, on, K);
}

// Sequences without tokens: their state (or its gradient) passes through.
__global__ void __launch_bounds__(256) scan_empty(ScanArgs a, const float *from, float *to)
{
    const int64_t C = (int64_t)a.H * a.D, n = blockIdx.x;
    if (a.cu ? a.cu[n] != a.cu[n + 1] : a.T != 0)
        return;
    for (int64_t c = threadIdx.x; c < C; c += 256)
        to[n * C + c] = from ? from[n * C + c] : 0.f;
}

cudaError_t pass_empty(const ScanArgs &a, const float *from, float *to, cudaStream_t s)
{
    if (!to || !a.some_empty)
        return cudaSuccess;
    scan_empty<<<(unsigned)a.N, 256, 0, s>>>(a, from, to);
    note_launch();
    return cudaGetLastError();
}

// Whether a thread walks a sequence alone, by the times that were measured (us):
// alone 0.25 a token of the longest, teams 2.2 a tile of the 608 at once, both
// no faster than HBM (64 rows of 16 tokens, 4096 channels, forward: 10 against
// 19; 4 rows of 100: 27 against 8).  Only where that costs little: ScanArgs::
// states has a state for each SCAN_BLOCK tokens then.  By the sizes alone, with
// the 6 bytes a value of bf16's forward for all: the backward has to choose as its
// forward did.
bool serial(int64_t tiles, int64_t longest, int64_t tokens, int64_t C)
{
    if (longest > 8 * SCAN_TILE)
        return false;
    const double hbm = (double)tokens * C * 6 / 5e6;
    const double alone = 0.25 * longest + hbm;
    const double teams = 2.0 + std::max(2.2 * tiles * ((C + CT - 1) / CT) / 608, hbm);
    return alone < teams;
}

PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        cudaDriverEntryPointQueryResult q;
        void *p = nullptr;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    });
    return fn;
}

// false: the layout is beyond a tensor map.
bool box_of(CUtensorMap *m, const ScanArgs &a, const Tok &x, int bf16, bool flat)
{
    const auto fn = encoder();
    const int64_t size = bf16 ? 2 : 4, lim = (int64_t)1 << 38;
    if (!fn || (!flat && a.D % CT))
        return false;
    const int64_t C = (int64_t)a.H * a.D;
    // a dimension of extent 1 never moves, any legal stride will do
    const int64_t sh = flat ? C : x.sh, st = a.T > 1 ? x.st : C, sb = a.B > 1 ? x.sb : C;
    if (sh <= 0 || st <= 0 || sb <= 0 || sh > lim || st > lim || sb > lim)
        return false;
    const cuuint64_t dims[4] = {(cuuint64_t)(flat ? C : a.D), (cuuint64_t)(flat ? 1 : a.H),
                                (cuuint64_t)a.T, (cuuint64_t)a.B};
    const cuuint64_t strides[3] = {(cuuint64_t)((sh * size + 15) / 16 * 16),
                                   (cuuint64_t)((st * size + 15) / 16 * 16),
                                   (cuuint64_t)((sb * size + 15) / 16 * 16)};
    const cuuint32_t box[4] = {(cuuint32_t)CT, 1, (cuuint32_t)SCAN_TILE, 1};
    const cuuint32_t one[4] = {1, 1, 1, 1};
    return fn(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4,
              const_cast<void *>(x.p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

cudaError_t sms_of(int *sms)
{
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 64 && (*sms = known[dev].load()) > 0)
        return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < 64)
        known[dev].store(*sms);
    return e;
}

// Launches the kernel, whose shared memory is set up on the first call per device.
template <bool BACK, typename T, typename TG, bool VEC, bool FLIP, bool GROUPED>
cudaError_t tiles(const ScanArgs &a, const Plan &k, const Boxes &boxes, int grid, cudaStream_t s)
{
    constexpr auto kernel = BACK ? scan_bwd_tiles<T, TG, VEC, FLIP, GROUPED>
                                 : scan_fwd_tiles<T, TG, VEC, FLIP, GROUPED>;
    static std::atomic<uint64_t> known;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev > 63 || !(known.load() >> dev & 1)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, RING);
        if (e != cudaSuccess)
            return e;
        if (dev < 64)
            known.fetch_or((uint64_t)1 << dev);
    }
    kernel<<<grid, CTA, RING, s>>>(a, k, boxes);
    note_launch();
    return cudaGetLastError();
}

template <bool BACK, typename T, typename TG, bool VEC, bool FLIP>
cudaError_t run(const ScanArgs &a, Plan k, void *ws, cudaStream_t s)
{
    constexpr int teams = BACK ? Bwd::TEAMS : Fwd::TEAMS;
    int sms = 0;
    cudaError_t e = sms_of(&sms);
    if (e != cudaSuccess)
        return e;
    // Chains: sequences x parts of the channels.  Few: segments, as many as there
    // are teams for, unless the maps that a segment starts from cost more than its
    // tiles (0.1 us a map, 4 us a tile for both passes: best at 7 sqrt(run)).
    // More: several teams for one chain, a unit to a group.  The measured border
    // (64 tiles a chain, us, segments and groups): forward 32 chains 33 and 62, 64
    // chains 56 and 63, 128 chains 106 and 68; backward 64 chains 107 and 133, 128
    // chains 182 and 134.
    const int64_t chains = (int64_t)a.N * k.parts;
    const int64_t slots = std::min<int64_t>((int64_t)sms * teams, MAX_UNITS);
    const int64_t run = (a.longest + SCAN_TILE - 1) / SCAN_TILE;
    int64_t segments = 1;
    if (BACK ? 7 * chains <= 4 * sms : 5 * chains <= 2 * sms)
        segments = std::min<int64_t>(
            {slots / chains, run, (int64_t)(7.0 * std::sqrt((double)run)), MAX_SEGMENTS});
    k.segments = (int)std::max<int64_t>(segments, 1);
    if (chains * k.segments > 0x7f000000)   // (a team steps beyond the last unit)
        return cudaErrorNotSupported;
    k.units = (int)(chains * k.segments);
    const int grid = (int)std::min<int64_t>(k.units, sms);
    k.group = 1;
    while (k.segments == 1 && k.group < teams && chains * k.group * 2 <= slots)
        k.group *= 2;
    Boxes boxes{};
    k.boxed = VEC && box_of(&boxes.x, a, a.x, a.bf16, k.flat) &&
              box_of(&boxes.g, a, a.g, a.gate_bf16, k.flat) &&
              (!BACK || box_of(&boxes.d, a, a.d_o, a.bf16, k.flat));
    if (k.segments > 1) {
        k.maps = static_cast<float2 *>(ws);
        k.map = 1;
        if ((e = tiles<BACK, T, TG, VEC, FLIP, false>(a, k, boxes, grid, s)) != cudaSuccess)
            return e;
        k.map = 0;
    }
    k.withhold = take_withheld();
    return k.group > 1 ? tiles<BACK, T, TG, VEC, FLIP, true>(a, k, boxes, grid, s)
                       : tiles<BACK, T, TG, VEC, FLIP, false>(a, k, boxes, grid, s);
}

// The tensors' rows are in whole 16-byte pieces: wide accesses and copies.  Of
// tensors whose heads are D apart (flat) all heads' channels are one row.
template <typename TT> bool wide(const TT &t, int bf16, bool flat, int64_t C, int D)
{
    const int n = bf16 ? 8 : 4;
    return reinterpret_cast<uintptr_t>(t.p) % 16 == 0 && t.sb % n == 0 && t.st % n == 0 &&
           (flat ? C % n == 0 : D % n == 0 && t.sh % n == 0);
}

template <bool BACK, typename T, typename TG>
cudaError_t launch(const ScanArgs &a, void *ws, cudaStream_t s)
{
    const int64_t C = (int64_t)a.H * a.D;
    // (one head's distance is not used)
    const int64_t sh[5] = {a.x.sh, a.g.sh, BACK ? a.d_o.sh : a.D, BACK ? a.dx.sh : a.D,
                           BACK ? a.dg.sh : a.o.p ? a.o.sh : a.D};
    const int64_t st[6] = {a.x.st, a.g.st, a.d_o.st, a.dx.st, a.dg.st, a.o.st};
    Plan k{};
    k.parts = (int)((C + CT - 1) / CT);
    k.flat = 1;
    for (int64_t v : sh)
        k.flat &= a.H == 1 || v == a.D;
    k.small = 1;
    for (int64_t v : st)
        k.small &= v <= (1 << 24);
    auto fits = [&](const auto &t, int bf16) { return wide(t, bf16, k.flat, C, a.D); };
    const bool vec = fits(a.x, a.bf16) && fits(a.g, a.gate_bf16) &&
                     (BACK ? fits(a.d_o, a.bf16) && fits(a.dx, a.bf16) && fits(a.dg, a.gate_bf16)
                           : !a.o.p || fits(a.o, a.bf16));
    if (a.serial) {
        const int64_t ctas = (a.N * ((C + V - 1) / V) + 127) / 128;
        if (ctas > 0x7fffffff)
            return cudaErrorNotSupported;
        if (BACK && vec)
            scan_bwd_serial<T, TG, true><<<(unsigned)ctas, 128, 0, s>>>(a, k.flat);
        else if (BACK)
            scan_bwd_serial<T, TG, false><<<(unsigned)ctas, 128, 0, s>>>(a, k.flat);
        else if (vec)
            scan_fwd_serial<T, TG, true><<<(unsigned)ctas, 128, 0, s>>>(a, k.flat);
        else
            scan_fwd_serial<T, TG, false><<<(unsigned)ctas, 128, 0, s>>>(a, k.flat);
        note_launch();
        return cudaGetLastError();
    }
    if (!vec)
        return run<BACK, T, TG, false, false>(a, k, ws, s);
    return a.reverse ? run<BACK, T, TG, true, true>(a, k, ws, s)
                     : run<BACK, T, TG, true, false>(a, k, ws, s);
}

template <bool BACK> cudaError_t dispatch(const ScanArgs &a, void *ws, cudaStream_t s)
{
    using bf = __nv_bfloat16;
    if ((int64_t)a.B * a.T == 0)
        return cudaSuccess;
    if (a.bf16 && a.gate_bf16)
        return launch<BACK, bf, bf>(a, ws, s);
    if (a.bf16)
        return launch<BACK, bf, float>(a, ws, s);
    return launch<BACK, float, float>(a, ws, s);
}

}  // namespace

void scan_plan(ScanArgs *a, int64_t tiles, int64_t longest)
{
    a->longest = longest;
    a->serial = serial(tiles, longest, (int64_t)a->B * a->T, (int64_t)a->H * a->D) &&
                (!a->cu || (int64_t)a->T <= (int64_t)a->N * SCAN_TILE);
}

size_t scan_states_bytes(int B, int T, int N, int H, int D)
{
    const int64_t C = (int64_t)H * D;
    auto blocks = [&](int64_t rows, int64_t size) { return rows * ((T + size - 1) / size); };
    // dense: B rows of T tokens
    const bool alone = serial(blocks(B, SCAN_TILE), T, (int64_t)B * T, C);
    const int64_t size = alone ? SCAN_BLOCK : SCAN_TILE;
    int64_t n = T <= size ? 0 : blocks(B, size);
    // packed: the lengths are not known, so for either kernel
    if (B == 1 && N > 0) {
        n = std::max(n, (int64_t)T / SCAN_TILE + N);
        if ((int64_t)T <= (int64_t)N * SCAN_TILE)
            n = std::max(n, (int64_t)T / SCAN_BLOCK + N);
    }
    return (size_t)n * C * sizeof(float);
}

size_t scan_maps_bytes(int T)
{
    return T > SCAN_TILE ? (size_t)MAX_UNITS * CT * sizeof(float2) : 0;
}

cudaError_t scan_forward(const ScanArgs &a, void *ws, cudaStream_t s)
{
    cudaError_t e = dispatch<false>(a, ws, s);
    return e != cudaSuccess ? e : pass_empty(a, a.init, a.fin, s);
}

cudaError_t scan_backward(const ScanArgs &a, void *ws, cudaStream_t s)
{
    cudaError_t e = dispatch<true>(a, ws, s);
    return e != cudaSuccess ? e : pass_empty(a, a.dfin, a.dinit, s);
}

cudaError_t scan_read_and_clear_error(cudaStream_t s, int *err)
{
    int zero = 0;
    cudaError_t e =
        cudaMemcpyFromSymbolAsync(err, g_scan_error, sizeof(int), 0, cudaMemcpyDeviceToHost, s);
    if (e == cudaSuccess)
        e = cudaMemcpyToSymbolAsync(g_scan_error, &zero, sizeof(int), 0, cudaMemcpyHostToDevice,
                                    s);
    if (e == cudaSuccess)
        e = cudaStreamSynchronize(s);
    return e;
}

}  // namespace la
