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
// So the tokens are cut into tiles that run in parallel: a CTA takes a tile of
// SCAN_TILE tokens x CT channels, its 16 token groups compose their L tokens,
// the groups are composed through shared memory, and the state that enters the
// tile comes from the tiles before it (tile_carry below).  x, g (and do) are
// read once and o (dx, dg) written once, whatever the length.
// The CTAs are persistent; the next tile's tokens are copied to shared memory
// (cp.async, every thread into slots of its own) while the present one is
// composed and waits for its state.
//
// All rows form one axis of processing positions (la_internal.h), so short and
// packed sequences fill tiles like long ones.  A sequence's first token is a
// reset: what comes before it is dropped by a select, never multiplied by zero,
// so that a NaN or an infinity stays in its sequence.
//
// Bound: HBM, 6 (bf16 gate) or 8 bytes a value forward, 10 or 14 backward.

#include <atomic>
#include <cstdint>

#include <cuda_bf16.h>

#include "../../include/la.h"
#include "la_internal.h"

namespace la {
namespace {

constexpr int LANES = 16, V = 4;            // lanes over channels, channels per lane
constexpr int CT = LANES * V;               // channels of a tile
constexpr int L = 8;                        // tokens per thread
constexpr int THREADS = 256, WARPS = THREADS / 32;
constexpr int PARTS = THREADS / CT;         // threads per channel in join
constexpr int EACH_WARPS = WARPS / PARTS;   // warps' maps per thread there
constexpr int GROUP = 32;                   // tiles per group of tile_carry
constexpr int EACH = GROUP / PARTS;
constexpr int ROW = CT + 4;                 // floats a warp's row takes: no bank conflicts in join
static_assert(THREADS / LANES * L == SCAN_TILE && PARTS == 4 && EACH_WARPS == 2, "tile shape");

constexpr unsigned long long EMPTY = ~0ull;   // an unwritten (A, B): see pack
constexpr unsigned long long WAIT_NS = 2000000000ull;
constexpr unsigned ALL = 0xffffffffu;

// LA_ERR_TIMEOUT when a tile waited in vain (la_get_device_error).
__device__ int g_scan_error;

// ---- arithmetic -------------------------------------------------------------
// The kernels are as near to the issue rate as to HBM, so the channels go
// through the packed fp32 instructions two at a time.

struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b)
{
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 f2(float a) { return f2(a, a); }
__device__ __forceinline__ float2 un(F2 a)
{
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c)
{
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b)
{
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b)
{
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
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
// 8192 tokens against 2e-6.  Larger |g| forget within four tokens; there 2^x
// is within 2^-22.
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
// an infinite state stays infinite, as it does token by token.
__device__ __forceinline__ float times(float a, float b)
{
    const float r = a * b;
    return r == 0.f && a != 0.f && b != 0.f ? 1.4e-45f : r;
}
__device__ __forceinline__ Val times(const Val &x, const Val &y)
{
    const float4 a = x.f(), b = y.f();
    return val(times(a.x, b.x), times(a.y, b.y), times(a.z, b.z), times(a.w, b.w));
}
// The state after tokens with the map (A, B); r: a sequence starts among them
// (what came before is dropped, A is not used).
__device__ __forceinline__ float through(float A, float B, int r, float s)
{
    return r ? B : fmaf(A, s, B);
}
__device__ __forceinline__ Val through(const Val &A, const Val &B, int r, const Val &s)
{
    return r ? B : fma2(A, s, B);
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

// Where a thread's channels are: head and channel of each.
template <bool VEC> struct Where {
    static constexpr int N = VEC ? 1 : V;
    unsigned on;   // bit v: channel v is there
    unsigned h[N], d[N];
    __device__ Where(unsigned c0, int lane, unsigned C, unsigned D) : on(0)
    {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const unsigned c = c0 + local_channel<VEC>(lane, v);
            on |= (c < C ? 1u : 0u) << v;
            if (v < N) {
                const unsigned k = c < C ? c : 0;   // not accessed
                h[v] = k / D;
                d[v] = k - h[v] * D;
            }
        }
    }
};

// One token tensor as a thread sees it, at one token's row.
template <typename T, bool VEC> struct Col {
    T *q;
    int64_t off[VEC ? 1 : V];
    __device__ Col(const Where<VEC> &w, const void *base, int64_t sh)
        : q(const_cast<T *>(static_cast<const T *>(base)))
    {
        if constexpr (VEC) {
            q += w.h[0] * sh + w.d[0];
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                off[v] = w.h[v] * sh + w.d[v];
        }
    }
    // the row's values to the thread's slot: asynchronously where they are wide
    __device__ void fetch(const T *r, unsigned on, Four<T> *slot) const
    {
        if constexpr (VEC) {
            const unsigned to = (unsigned)__cvta_generic_to_shared(slot);
            if constexpr (sizeof(*slot) == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(r)
                             : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(r)
                             : "memory");
        } else {
            float f[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                f[v] = on >> v & 1 ? ldt(r + off[v]) : 0.f;
            slot->set(val(f[0], f[1], f[2], f[3]));
        }
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

// The tile's tokens: (batch row, token) and the number of the sequence.
struct Tokens {
    int2 at[SCAN_TILE];
    int seq[SCAN_TILE];
};

// Walks the rows of a tensor over a group's tokens, up or down.  step: the
// tokens are neighbours in one batch row (else each is looked up).
template <typename T, bool VEC> struct Walk {
    const Col<T, VEC> &col;
    const int2 *at;
    int64_t sb, st, by;
    bool step;
    T *r;
    __device__ Walk(const Col<T, VEC> &c, const int2 *tokens, int64_t sb_, int64_t st_, int first,
                    int reverse, bool down, bool step_)
        : col(c), at(tokens), sb(sb_), st(st_), by((reverse != 0) != down ? -st_ : st_),
          step(step_), r(row(first))
    {
    }
    __device__ T *row(int e) const { return col.q + at[e].x * sb + at[e].y * st; }
    __device__ void to(int e)   // from e - 1 (up) or e + 1 (down)
    {
        r += by;
        if (!step)
            r = row(e);
    }
};

struct Marks {
    unsigned starts, ends;   // bit e: the group's token e is its sequence's first, last
};

__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// All but the newest group of the thread's copies have landed.
__device__ __forceinline__ void copies_before_last()
{
    asm volatile("cp.async.wait_group 1;" ::: "memory");
}

// Fills the table of the warp's 2 L tokens from position q on (its lanes below
// 2 L take one each).  *edge: where the lane's sequence begins (LAST: its last
// position).
template <bool LAST>
__device__ __forceinline__ Marks look_up(const ScanArgs &a, Tokens &tk, int64_t P, int64_t q,
                                         int64_t *edge)
{
    const int lane = threadIdx.x % 32, slot = threadIdx.x / 32 * 2 * L + lane;
    bool start = false, end = false;
    const int64_t p = q + lane;
    if (lane < 2 * L && p < P) {
        int b = 0, t, n;
        if (a.cu) {
            t = (int)(a.reverse ? a.T - 1 - p : p);
            n = 0;
            for (int hi = a.N; hi - n > 1;) {   // cu[n] <= t < cu[hi]
                const int m = (n + hi) / 2;
                if (a.cu[m] <= t)
                    n = m;
                else
                    hi = m;
            }
            const int lo = a.cu[n], hi = a.cu[n + 1];
            start = t == (a.reverse ? hi - 1 : lo);
            end = t == (a.reverse ? lo : hi - 1);
            *edge = p + (LAST ? (a.reverse ? t - lo : hi - 1 - t)
                              : (a.reverse ? t - hi + 1 : lo - t));
        } else {
            int j;
            if (P <= 0x7fffffff) {
                b = (int)((unsigned)p / (unsigned)a.T);
                j = (int)((unsigned)p - (unsigned)b * (unsigned)a.T);
            } else {
                b = (int)(p / a.T);
                j = (int)(p - (int64_t)b * a.T);
            }
            t = a.reverse ? a.T - 1 - j : j;
            n = b;
            start = j == 0;
            end = j == a.T - 1;
            *edge = p + (LAST ? a.T - 1 - j : -j);
        }
        tk.at[slot] = make_int2(b, t);
        tk.seq[slot] = n;
    }
    const unsigned ss = __ballot_sync(ALL, start), es = __ballot_sync(ALL, end);
    __syncwarp();
    const int shift = lane / LANES * L;
    return Marks{ss >> shift & ((1u << L) - 1), es >> shift & ((1u << L) - 1)};
}

// A state vector's values at the thread's channels (0 where absent).
template <bool VEC>
__device__ __forceinline__ Val get_state(const float *from, int64_t n, int64_t C, unsigned c0,
                                         int lane, unsigned on)
{
    float s[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        s[v] = from && (on >> v & 1) ? from[n * C + c0 + local_channel<VEC>(lane, v)] : 0.f;
    return val(s[0], s[1], s[2], s[3]);
}
template <bool VEC>
__device__ __forceinline__ void put_state(float *to, int64_t n, int64_t C, unsigned c0, int lane,
                                          unsigned on, const Val &x)
{
    const float4 f = x.f();
    float *p = to + n * C + c0;
    if (on & 1)
        p[local_channel<VEC>(lane, 0)] = f.x;
    if (on & 2)
        p[local_channel<VEC>(lane, 1)] = f.y;
    if (on & 4)
        p[local_channel<VEC>(lane, 2)] = f.z;
    if (on & 8)
        p[local_channel<VEC>(lane, 3)] = f.w;
}

// ---- the state that enters a tile --------------------------------------------

struct Link {
    unsigned *head;              // [0] the next item, [1] cleared when a wait ran out
    unsigned long long *agg;     // [tile][C]: the tile's own (A, B)
    unsigned long long *inc;     // [group][C]: the state after the group's last tile
    int tiles;                   // along the tokens
    int parts;                   // along the channels
    int withhold;                // diagnostic: the first tile does not publish
};

__device__ __forceinline__ void publish(unsigned long long *p, float A, float B)
{
    unsigned a = __float_as_uint(A);
    if (a == 0xffffffffu)   // a NaN that would read as EMPTY
        a = 0x7fffffffu;
    const unsigned long long v = (unsigned long long)a << 32 | __float_as_uint(B);
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}
__device__ __forceinline__ unsigned long long peek(const unsigned long long *p)
{
    unsigned long long v;
    asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ unsigned long long now_ns()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// One round of a wait that began at t0: true when it has to end, after WAIT_NS
// (which raises the error word and the call's own flag) or because another wait
// of the call ended so.
__device__ __forceinline__ bool give_up(const Link &k, unsigned long long &t0)
{
    volatile unsigned *flag = k.head + 1;
    if (*flag == 0)
        return true;
    const unsigned long long t = now_ns();
    if (!t0)
        t0 = t;
    if (t - t0 <= WAIT_NS) {
        __nanosleep(100);   // leave the issue slots to the warps that compute
        return false;
    }
    *flag = 0;
    atomicExch(&g_scan_error, LA_ERR_TIMEOUT);
    return true;
}

// The state that enters tile m (tiles numbered in the order of the chain, ms
// the tile in which its sequence starts, ms < m) at channel c, by the PARTS
// neighbouring lanes of that channel.
//
// Tiles come in groups of GROUP.  The state is composed from the maps of the
// group's tiles before m and, where the sequence started before the group,
// from the state after the previous group, which that group's last tile
// publishes.  The maps need no other tile, so they are there as soon as their
// tiles are loaded: the chain proceeds a group, not a tile, at a time (one hop
// is one to two microseconds; 2048 tiles of a sequence of 262144 tokens one
// after the other would take milliseconds).  What is composed with what depends
// on the tiles' numbers alone, never on which tile came first, so results
// repeat bit for bit.  A value and its readiness are one 64-bit word: no fence,
// no second read.
__device__ __forceinline__ float tile_carry(const Link &k, int64_t C, unsigned c, int m, int ms)
{
    const int part = threadIdx.x % PARTS;
    const bool on = c < C;
    const int gs = m / GROUP * GROUP;
    const bool far = ms < gs;
    const int first = far ? gs : ms + 1, each = (m - first + PARTS - 1) / PARTS;
    const int lo = first + part * each;
    const unsigned long long *ag = k.agg + c + (int64_t)lo * C;
    const unsigned long long *bp =
        far ? k.inc + (int64_t)(m / GROUP - 1) * C + c : k.agg + c + (int64_t)ms * C;
    const int n = on ? min(each, m - lo) : 0;   // the thread's tiles
    unsigned long long v[EACH], b = on && part == 0 ? EMPTY : 0, t0 = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i)
        v[i] = i < n ? EMPTY : 0;
    for (;;) {
        bool all = true;
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            if (v[i] == EMPTY)
                v[i] = peek(ag + i * C);
        if (b == EMPTY)
            b = peek(bp);
#pragma unroll
        for (int i = 0; i < EACH; ++i)
            all &= v[i] != EMPTY;
        if ((all && b != EMPTY) || give_up(k, t0))
            break;
    }
    float A = 1.f, B = 0.f;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        if (i < n) {
            const float a2 = __uint_as_float((unsigned)(v[i] >> 32));
            B = fmaf(a2, B, __uint_as_float((unsigned)v[i]));
            A = times(A, a2);
        }
    }
    __syncwarp();
#pragma unroll
    for (int i = 1; i < PARTS; i *= 2) {
        const float a2 = __shfl_down_sync(ALL, A, i), b2 = __shfl_down_sync(ALL, B, i);
        B = fmaf(a2, B, b2);   // (of the lanes whose part is a multiple of 2 i)
        A = times(A, a2);
    }
    const float s = fmaf(A, __uint_as_float((unsigned)b), B);
    return __shfl_sync(ALL, s, threadIdx.x % 32 / PARTS * PARTS);
}

struct Shared {
    float A[WARPS][ROW], B[WARPS][ROW];   // the warps' maps
    float fB[WARPS][ROW];                 // backward: B of their forward maps (A is the same)
    float S[WARPS][ROW], fS[WARPS][ROW];  // the state that enters the warp
    int reset[WARPS], freset[WARPS];      // whether a sequence starts in the warp's tokens
    Tokens tk[2];                         // by stage, as the next two
    int64_t edge[2];                      // where the chain's sequence began (its position)
    int entered[2];                       // backward: the forward chain enters the tile
    unsigned item;                        // the one after the present one
};

// What PARTS neighbouring lanes know of a channel's maps: part p holds those of
// the warps 2p and 2p + 1 in the order of the chain (BACK: warp 7 first).
struct Run {
    float A0, B0;   // the first warp's map
    int r0;
    float eA, eB;   // the map of all warps before it
    int er;
    float A, B;     // the map of the tile (in every lane)
    int r;
};
template <bool BACK>
__device__ __forceinline__ Run run_of(const float (&A)[WARPS][ROW], const float (&B)[WARPS][ROW],
                                      const int (&reset)[WARPS])
{
    const int c = threadIdx.x / PARTS, part = threadIdx.x % PARTS;
    const int w0 = BACK ? WARPS - 1 - 2 * part : 2 * part, w1 = BACK ? w0 - 1 : w0 + 1;
    Run q;
    q.A0 = A[w0][c];
    q.B0 = B[w0][c];
    q.r0 = reset[w0];
    q.A = times(q.A0, A[w1][c]);
    q.B = through(A[w1][c], B[w1][c], reset[w1], q.B0);
    q.r = q.r0 | reset[w1];
#pragma unroll
    for (int i = 1; i < PARTS; i *= 2) {
        const float a = __shfl_up_sync(ALL, q.A, i), b = __shfl_up_sync(ALL, q.B, i);
        const int r = __shfl_up_sync(ALL, q.r, i);
        if (part >= i) {
            q.B = through(q.A, q.B, q.r, b);
            q.A = times(q.A, a);
            q.r |= r;
        }
    }
    q.eA = __shfl_up_sync(ALL, q.A, 1);
    q.eB = __shfl_up_sync(ALL, q.B, 1);
    q.er = __shfl_up_sync(ALL, q.r, 1);
    if (part == 0)
        q.eA = 1.f, q.eB = 0.f, q.er = 0;
    const int last = threadIdx.x % 32 / PARTS * PARTS + PARTS - 1;
    q.A = __shfl_sync(ALL, q.A, last);
    q.B = __shfl_sync(ALL, q.B, last);
    q.r = __shfl_sync(ALL, q.r, last);
    return q;
}
// The states that enter the warps, from the one that enters the tile.
template <bool BACK>
__device__ __forceinline__ void spread(float (&S)[WARPS][ROW], const Run &q, float s)
{
    const int c = threadIdx.x / PARTS, part = threadIdx.x % PARTS;
    const int w0 = BACK ? WARPS - 1 - 2 * part : 2 * part, w1 = BACK ? w0 - 1 : w0 + 1;
    const float in = through(q.eA, q.eB, q.er, s);
    S[w0][c] = in;
    S[w1][c] = through(q.A0, q.B0, q.r0, in);
}

// Publishes the tile's map, waits for the state that enters it and hands it to
// the warps.  edge: where the chain's sequence began, in tiles; chained: before
// this tile.  Returns the entering state (at channel threadIdx.x / PARTS).
template <bool BACK>
__device__ __forceinline__ float join(const Link &k, Shared &sm, int64_t C, unsigned c0, int m,
                                      bool chained, int ms)
{
    const Run q = run_of<BACK>(sm.A, sm.B, sm.reset);
    const unsigned c = c0 + threadIdx.x / PARTS;
    const bool speaks = k.head && threadIdx.x % PARTS == 0 && c < C;
    if (speaks && !(k.withhold && m == 0))
        publish(k.agg + m * C + c, q.A, q.B);
    const float s = chained ? tile_carry(k, C, c, m, ms) : 0.f;
    if (speaks && m % GROUP == GROUP - 1)
        publish(k.inc + m / GROUP * C + c, 0.f, through(q.A, q.B, q.r, s));
    spread<BACK>(sm.S, q, s);
    return s;
}

// ---- tiles ------------------------------------------------------------------

// What a thread keeps of a tile whose copies it has issued.
struct Tile {
    unsigned item;
    int count;   // tokens of the thread's group
    Marks mk;
};

// The slots of a stage: [token of the group][thread].
template <typename T> __device__ __forceinline__ Four<T> *slots(uint8_t *base)
{
    return reinterpret_cast<Four<T> *>(base) + threadIdx.x;
}
template <typename T> constexpr int slot_bytes() { return L * THREADS * (int)sizeof(Four<T>); }
template <bool BACK, typename T, typename TG> constexpr int stage_bytes()
{
    return slot_bytes<T>() * (BACK ? 2 : 1) + slot_bytes<TG>();
}

// Whether a group's tokens are neighbours in one batch row.
__device__ __forceinline__ bool in_step(const ScanArgs &a, const Marks &mk)
{
    return a.cu || !(mk.starts >> 1);
}

// Looks the tile's tokens up and issues the copies of x and g (BACK: and do).
template <bool BACK, typename T, typename TG, bool VEC>
__device__ __forceinline__ Tile issue(const ScanArgs &a, const Link &k, Shared &sm,
                                      uint8_t *stage, int st, unsigned item, int64_t C, int64_t P)
{
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES, warp = threadIdx.x / 32;
    Tile t{item, 0, Marks{0, 0}};
    if (item >= (unsigned)k.tiles * (unsigned)k.parts)
        return t;
    const unsigned m = item / (unsigned)k.parts, c0 = (item - m * (unsigned)k.parts) * CT;
    const int64_t p0 = (int64_t)(BACK ? k.tiles - 1 - (int)m : (int)m) * SCAN_TILE;
    const Where<VEC> w(c0, lane, (unsigned)C, (unsigned)a.D);
    t.count = w.on ? (int)max((int64_t)0, min((int64_t)L, P - p0 - group * L)) : 0;
    int64_t edge = 0;
    t.mk = look_up<BACK>(a, sm.tk[st], P, p0 + warp * 2 * L, &edge);
    if (BACK) {
        const int l = threadIdx.x % 32;   // the lane of the tile's last position
        if (l < 2 * L && p0 + warp * 2 * L + l == min(P, p0 + SCAN_TILE) - 1)
            sm.edge[st] = edge;
        if (threadIdx.x == 0)
            sm.entered[st] = !(t.mk.starts & 1);
    } else if (threadIdx.x == 0) {
        sm.edge[st] = edge;
    }
    if (t.count) {
        const int2 *at = sm.tk[st].at + group * L;
        const bool step = in_step(a, t.mk);
        const Col<T, VEC> xc(w, a.x.p, a.x.sh), dc(w, a.d_o.p, a.d_o.sh);
        const Col<TG, VEC> gc(w, a.g.p, a.g.sh);
        Walk<T, VEC> x(xc, at, a.x.sb, a.x.st, 0, a.reverse, false, step);
        Walk<T, VEC> d(dc, at, a.d_o.sb, a.d_o.st, 0, a.reverse, false, step);
        Walk<TG, VEC> g(gc, at, a.g.sb, a.g.st, 0, a.reverse, false, step);
        Four<T> *xs = slots<T>(stage), *ds = slots<T>(stage + slot_bytes<T>() + slot_bytes<TG>());
        Four<TG> *gs = slots<TG>(stage + slot_bytes<T>());
#pragma unroll
        for (int e = 0; e < L; ++e) {
            if (e < t.count) {
                if (e) {
                    x.to(e);
                    g.to(e);
                    if (BACK)
                        d.to(e);
                }
                xc.fetch(x.r, w.on, xs + e * THREADS);
                gc.fetch(g.r, w.on, gs + e * THREADS);
                if (BACK)
                    dc.fetch(d.r, w.on, ds + e * THREADS);
            }
        }
    }
    return t;
}

// The CTA's items: taken in the order of the chain, so that whatever a tile
// waits for is held by a CTA that runs and has nothing before it to wait for.
__device__ __forceinline__ unsigned take(const Link &k)
{
    return atomicAdd(k.head, 1u) + 1u;   // the counter starts at -1
}

// ---- forward ----------------------------------------------------------------

template <typename T, typename TG, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) scan_fwd_tiles(const ScanArgs a, const Link k)
{
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ Shared sm;
    const int64_t C = (int64_t)a.H * a.D, P = (int64_t)a.B * a.T;
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES * L;
    const int warp = threadIdx.x / 32;
    const bool odd = threadIdx.x & LANES;   // the second group of the warp
    const unsigned items = (unsigned)k.tiles * (unsigned)k.parts;
    constexpr int STAGE = stage_bytes<false, T, TG>();
    if (threadIdx.x == 0)
        sm.item = k.head ? take(k) : blockIdx.x;
    __syncthreads();
    Tile cur = issue<false, T, TG, VEC>(a, k, sm, ring, 0, sm.item, C, P);
    copies_issued();
    __syncthreads();
    if (threadIdx.x == 0)
        sm.item = k.head ? take(k) : items;
    for (int st = 0; cur.item < items; st ^= 1) {
        __syncthreads();
        const Tile nxt = issue<false, T, TG, VEC>(a, k, sm, ring + (st ^ 1) * STAGE, st ^ 1,
                                                  sm.item, C, P);
        copies_issued();
        unsigned after = items;
        if (threadIdx.x == 0 && k.head && nxt.item < items)
            after = take(k);
        copies_before_last();
        const Tokens &tk = sm.tk[st];
        const Four<T> *xs = slots<T>(ring + st * STAGE);
        const Four<TG> *gs = slots<TG>(ring + st * STAGE + slot_bytes<T>());
        const unsigned tile = cur.item / (unsigned)k.parts;
        const unsigned c0 = (cur.item - tile * (unsigned)k.parts) * CT;
        const Where<VEC> w(c0, lane, (unsigned)C, (unsigned)a.D);
        const Marks mk = cur.mk;
        const int count = cur.count;
        const bool plain = count == L && !(mk.starts | mk.ends);
        // the thread's tokens composed to s -> A s + B; their decays are kept
        Val d[L], A = val(1.f, 1.f, 1.f, 1.f), B = val(0.f, 0.f, 0.f, 0.f);
        if (plain) {
#pragma unroll
            for (int e = 0; e < L; ++e) {
                d[e] = decay(gs[e * THREADS].get());
                B = fma2(d[e], B, xs[e * THREADS].get());
                A = mul2(A, d[e]);
            }
        } else {
#pragma unroll
            for (int e = 0; e < L; ++e) {
                if (e < count) {
                    if (mk.starts >> e & 1)   // from here on A is not used
                        B = get_state<VEC>(a.init, tk.seq[slot + e], C, c0, lane, w.on);
                    d[e] = decay(gs[e * THREADS].get());
                    B = fma2(d[e], B, xs[e * THREADS].get());
                    A = mul2(A, d[e]);
                }
            }
        }
        // the two groups of a warp, then the warps
        const int r = mk.starts != 0, er = __shfl_xor_sync(ALL, r, LANES);
        const Val eA = shuffled(A), eB = shuffled(B);   // the other group's map
        if (odd) {
            put_row<VEC>(sm.A[warp], lane, times(A, eA));
            put_row<VEC>(sm.B[warp], lane, through(A, B, r, eB));
            if (lane == 0)
                sm.reset[warp] = r | er;
        }
        __syncthreads();
        const int64_t edge = sm.edge[st];
        const bool chained = (int64_t)tile * SCAN_TILE > edge;   // goes on with an earlier state
        const float in =
            join<false>(k, sm, C, c0, (int)tile, chained, (int)(edge / SCAN_TILE));
        if (a.states && chained && threadIdx.x % PARTS == 0 && c0 + threadIdx.x / PARTS < C)
            a.states[tile * C + c0 + threadIdx.x / PARTS] = in;
        __syncthreads();
        if (count && (a.o.p || a.fin)) {
            Val s = get_row<VEC>(sm.S[warp], lane);
            if (odd)
                s = through(eA, eB, er, s);
            const Col<T, VEC> oc(w, a.o.p, a.o.sh);
            Walk<T, VEC> o(oc, tk.at + slot, a.o.sb, a.o.st, 0, a.reverse, false,
                           in_step(a, mk));
            if (plain && a.o.p) {
#pragma unroll
                for (int e = 0; e < L; ++e) {
                    s = fma2(d[e], s, xs[e * THREADS].get());
                    if (e)
                        o.to(e);
                    oc.store(o.r, w.on, s);
                }
            } else {
#pragma unroll
                for (int e = 0; e < L; ++e) {
                    if (e < count) {
                        if (mk.starts >> e & 1)
                            s = get_state<VEC>(a.init, tk.seq[slot + e], C, c0, lane, w.on);
                        s = fma2(d[e], s, xs[e * THREADS].get());
                        if (e)
                            o.to(e);
                        if (a.o.p)
                            oc.store(o.r, w.on, s);
                        if (a.fin && (mk.ends >> e & 1))
                            put_state<VEC>(a.fin, tk.seq[slot + e], C, c0, lane, w.on, s);
                    }
                }
            }
        }
        cur = nxt;
        if (threadIdx.x == 0)
            sm.item = after;
    }
}

// ---- backward -----------------------------------------------------------------
// The chain runs from the last position to the first; s_{t-1} comes from the
// states that entered the tiles in the forward.

template <typename T, typename TG, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) scan_bwd_tiles(const ScanArgs a, const Link k)
{
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ Shared sm;
    const int64_t C = (int64_t)a.H * a.D, P = (int64_t)a.B * a.T;
    const int lane = threadIdx.x % LANES, slot = threadIdx.x / LANES * L;
    const int warp = threadIdx.x / 32;
    const bool odd = threadIdx.x & LANES;
    const unsigned items = (unsigned)k.tiles * (unsigned)k.parts;
    constexpr int STAGE = stage_bytes<true, T, TG>();
    if (threadIdx.x == 0)
        sm.item = k.head ? take(k) : blockIdx.x;
    __syncthreads();
    Tile cur = issue<true, T, TG, VEC>(a, k, sm, ring, 0, sm.item, C, P);
    copies_issued();
    __syncthreads();
    if (threadIdx.x == 0)
        sm.item = k.head ? take(k) : items;
    for (int st = 0; cur.item < items; st ^= 1) {
        __syncthreads();
        const Tile nxt = issue<true, T, TG, VEC>(a, k, sm, ring + (st ^ 1) * STAGE, st ^ 1,
                                                 sm.item, C, P);
        copies_issued();
        unsigned after = items;
        if (threadIdx.x == 0 && k.head && nxt.item < items)
            after = take(k);
        copies_before_last();
        const Tokens &tk = sm.tk[st];
        const Four<T> *xs = slots<T>(ring + st * STAGE);
        const Four<TG> *gs = slots<TG>(ring + st * STAGE + slot_bytes<T>());
        const Four<T> *ds = slots<T>(ring + st * STAGE + slot_bytes<T>() + slot_bytes<TG>());
        const unsigned m = cur.item / (unsigned)k.parts;
        const unsigned c0 = (cur.item - m * (unsigned)k.parts) * CT;
        const int tile = k.tiles - 1 - (int)m;
        const int64_t pe = min(P, (int64_t)(tile + 1) * SCAN_TILE) - 1;   // the last position
        const Where<VEC> w(c0, lane, (unsigned)C, (unsigned)a.D);
        const Marks mk = cur.mk;
        const int count = cur.count;
        const bool plain = count == L && !(mk.starts | mk.ends);
        // the thread's maps of the forward chain (A, fB) and of the backward
        // chain (A, B): the same decays, one product
        Val d[L], A = val(1.f, 1.f, 1.f, 1.f), B = val(0.f, 0.f, 0.f, 0.f), fB = B;
        if (plain) {
#pragma unroll
            for (int e = 0; e < L; ++e) {
                d[e] = decay(gs[e * THREADS].get());
                fB = fma2(d[e], fB, xs[e * THREADS].get());
                A = mul2(A, d[e]);
            }
#pragma unroll
            for (int e = L - 1; e >= 0; --e)
                B = mul2(d[e], add2(ds[e * THREADS].get(), B));
        } else {
#pragma unroll
            for (int e = 0; e < L; ++e) {
                if (e < count) {
                    if (mk.starts >> e & 1)
                        fB = get_state<VEC>(a.init, tk.seq[slot + e], C, c0, lane, w.on);
                    d[e] = decay(gs[e * THREADS].get());
                    fB = fma2(d[e], fB, xs[e * THREADS].get());
                    A = mul2(A, d[e]);
                }
            }
#pragma unroll
            for (int e = L - 1; e >= 0; --e) {
                if (e < count) {
                    if (mk.ends >> e & 1)
                        B = get_state<VEC>(a.dfin, tk.seq[slot + e], C, c0, lane, w.on);
                    B = mul2(d[e], add2(ds[e * THREADS].get(), B));
                }
            }
        }
        // the other group's maps: the even group's forward one for the odd, the
        // odd group's backward one for the even
        const int fr = mk.starts != 0, r = mk.ends != 0;
        const int orr = __shfl_xor_sync(ALL, odd ? r : fr, LANES);
        const Val oA = shuffled(A), oB = shuffled(odd ? B : fB);
        if (odd) {
            put_row<VEC>(sm.fB[warp], lane, through(A, fB, fr, oB));
            if (lane == 0)
                sm.freset[warp] = fr | orr;
        } else {
            put_row<VEC>(sm.A[warp], lane, times(A, oA));
            put_row<VEC>(sm.B[warp], lane, through(A, B, r, oB));
            if (lane == 0)
                sm.reset[warp] = r | orr;
        }
        __syncthreads();
        {
            // the forward states that enter the warps
            const unsigned c = c0 + threadIdx.x / PARTS;
            const float s = sm.entered[st] && c < C ? a.states[tile * C + c] : 0.f;
            spread<false>(sm.fS, run_of<false>(sm.A, sm.fB, sm.freset), s);
        }
        const int64_t edge = sm.edge[st];
        join<true>(k, sm, C, c0, (int)m, pe < edge, k.tiles - 1 - (int)(edge / SCAN_TILE));
        __syncthreads();
        if (count) {
            // the states before the thread's tokens
            Val x[L];
            {
                Val s = get_row<VEC>(sm.fS[warp], lane);
                if (odd)
                    s = through(oA, oB, orr, s);
#pragma unroll
                for (int e = 0; e < L; ++e) {
                    if (e < count) {
                        if (mk.starts >> e & 1)
                            s = get_state<VEC>(a.init, tk.seq[slot + e], C, c0, lane, w.on);
                        x[e] = s;
                        s = fma2(d[e], s, xs[e * THREADS].get());
                    }
                }
            }
            Val K = get_row<VEC>(sm.S[warp], lane);
            if (!odd)
                K = through(oA, oB, orr, K);
            const Col<T, VEC> dxc(w, a.dx.p, a.dx.sh);
            const Col<TG, VEC> dgc(w, a.dg.p, a.dg.sh);
            const bool step = in_step(a, mk);
            Walk<T, VEC> dx(dxc, tk.at + slot, a.dx.sb, a.dx.st, count - 1, a.reverse, true, step);
            Walk<TG, VEC> dg(dgc, tk.at + slot, a.dg.sb, a.dg.st, count - 1, a.reverse, true,
                             step);
#pragma unroll
            for (int e = L - 1; e >= 0; --e) {
                if (e < count) {
                    if (mk.ends >> e & 1)
                        K = get_state<VEC>(a.dfin, tk.seq[slot + e], C, c0, lane, w.on);
                    const Val G = add2(ds[e * THREADS].get(), K);
                    K = mul2(d[e], G);
                    if (e < count - 1) {
                        dx.to(e);
                        dg.to(e);
                    }
                    dxc.store(dx.r, w.on, G);
                    dgc.store(dg.r, w.on, mul2(K, x[e]));
                    if (a.dinit && (mk.starts >> e & 1))
                        put_state<VEC>(a.dinit, tk.seq[slot + e], C, c0, lane, w.on, K);
                }
            }
        }
        cur = nxt;
        if (threadIdx.x == 0)
            sm.item = after;
    }
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

bool wide(const void *p, int64_t sb, int64_t st, int64_t sh, int bf16)
{
    return reinterpret_cast<uintptr_t>(p) % (bf16 ? 8 : 16) == 0 && sb % V == 0 && st % V == 0 &&
           sh % V == 0;
}
bool wide(const Tok &t, int bf16) { return wide(t.p, t.sb, t.st, t.sh, bf16); }
bool wide(const TokOut &t, int bf16) { return wide(t.p, t.sb, t.st, t.sh, bf16); }

int64_t tiles_of(int64_t positions) { return (positions + SCAN_TILE - 1) / SCAN_TILE; }

size_t link_bytes(int64_t tiles, int64_t C)
{
    return 256 + (size_t)(tiles + (tiles + GROUP - 1) / GROUP) * C * sizeof(unsigned long long);
}

// CTAs of a kernel that the device holds at once; sets the kernel's shared
// memory up on the first call per device.
template <bool BACK, typename T, typename TG, bool VEC, typename K>
cudaError_t resident_of(K kernel, int smem, int *ctas)
{
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    if (dev < 64 && (*ctas = known[dev].load()) > 0)
        return cudaSuccess;
    int sms = 0, per = 0;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e == cudaSuccess)
        e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, THREADS, smem);
    if (e != cudaSuccess)
        return e;
    *ctas = sms * (per > 0 ? per : 1);
    if (dev < 64)
        known[dev].store(*ctas);
    return cudaSuccess;
}

template <bool BACK, typename T, typename TG, bool VEC>
cudaError_t run(const ScanArgs &a, const Link &k, int64_t grid, cudaStream_t s)
{
    constexpr auto kernel = BACK ? scan_bwd_tiles<T, TG, VEC> : scan_fwd_tiles<T, TG, VEC>;
    constexpr int smem = 2 * stage_bytes<BACK, T, TG>();
    int ctas = 0;
    cudaError_t e = resident_of<BACK, T, TG, VEC>(kernel, smem, &ctas);
    if (e != cudaSuccess)
        return e;
    if (k.head && grid > ctas)
        grid = ctas;
    kernel<<<(unsigned)grid, THREADS, smem, s>>>(a, k);
    note_launch();
    return cudaGetLastError();
}

template <typename T, typename TG, bool VEC>
cudaError_t launch(bool back, const ScanArgs &a, void *ws, cudaStream_t s)
{
    const int64_t C = (int64_t)a.H * a.D, tiles = tiles_of((int64_t)a.B * a.T);
    const int64_t parts = (C + CT - 1) / CT;
    if (tiles * parts > 0x7fffffff)
        return cudaErrorNotSupported;
    Link k{};
    k.tiles = (int)tiles;
    k.parts = (int)parts;
    const int64_t grid = tiles * parts;
    if (tiles > 1) {
        const size_t bytes = link_bytes(tiles, C);
        cudaError_t e = cudaMemsetAsync(ws, 0xff, bytes, s);
        if (e != cudaSuccess)
            return e;
        k.head = static_cast<unsigned *>(ws);
        k.agg = reinterpret_cast<unsigned long long *>(static_cast<uint8_t *>(ws) + 256);
        k.inc = k.agg + tiles * C;
        k.withhold = take_withheld();
    }
    return back ? run<true, T, TG, VEC>(a, k, grid, s) : run<false, T, TG, VEC>(a, k, grid, s);
}

cudaError_t dispatch(bool back, const ScanArgs &a, bool vec, void *ws, cudaStream_t s)
{
    using bf = __nv_bfloat16;
    if ((int64_t)a.B * a.T == 0)
        return cudaSuccess;
    if (a.bf16 && a.gate_bf16)
        return vec ? launch<bf, bf, true>(back, a, ws, s) : launch<bf, bf, false>(back, a, ws, s);
    if (a.bf16)
        return vec ? launch<bf, float, true>(back, a, ws, s)
                   : launch<bf, float, false>(back, a, ws, s);
    return vec ? launch<float, float, true>(back, a, ws, s)
               : launch<float, float, false>(back, a, ws, s);
}

}  // namespace

size_t scan_link_bytes(int B, int T, int H, int D)
{
    const int64_t tiles = tiles_of((int64_t)B * T);
    return tiles > 1 ? link_bytes(tiles, (int64_t)H * D) : 0;
}

cudaError_t scan_forward(const ScanArgs &a, void *ws, cudaStream_t s)
{
    const bool vec = a.D % V == 0 && wide(a.x, a.bf16) && wide(a.g, a.gate_bf16) &&
                     (!a.o.p || wide(a.o, a.bf16));
    cudaError_t e = dispatch(false, a, vec, ws, s);
    return e != cudaSuccess ? e : pass_empty(a, a.init, a.fin, s);
}

cudaError_t scan_backward(const ScanArgs &a, void *ws, cudaStream_t s)
{
    const bool vec = a.D % V == 0 && wide(a.x, a.bf16) && wide(a.g, a.gate_bf16) &&
                     wide(a.d_o, a.bf16) && wide(a.dx, a.bf16) && wide(a.dg, a.gate_bf16);
    cudaError_t e = dispatch(true, a, vec, ws, s);
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
