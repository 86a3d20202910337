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
constexpr int PARTS = THREADS / CT;         // threads per channel in tile_carry
constexpr int GROUP = 32;                   // tiles per group of tile_carry
constexpr int EACH = GROUP / PARTS;
static_assert(THREADS / LANES * L == SCAN_TILE, "tile shape");

constexpr unsigned long long EMPTY = ~0ull;   // an unwritten (A, B): see pack
constexpr unsigned long long WAIT_NS = 2000000000ull;

// LA_ERR_TIMEOUT when a tile waited in vain (la_get_device_error).
__device__ int g_scan_error;

// ---- types ----------------------------------------------------------------

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

// Four values as loaded: 8 bytes of bf16, 16 of fp32.
template <typename T> struct Four;
template <> struct Four<float> {
    float4 r;
    __device__ void get(float (&v)[V]) const
    {
        v[0] = r.x;
        v[1] = r.y;
        v[2] = r.z;
        v[3] = r.w;
    }
    __device__ void set(const float (&v)[V]) { r = make_float4(v[0], v[1], v[2], v[3]); }
};
template <> struct Four<__nv_bfloat16> {
    uint2 r;
    __device__ void get(float (&v)[V]) const
    {
        v[0] = __uint_as_float(r.x << 16);
        v[1] = __uint_as_float(r.x & 0xffff0000u);
        v[2] = __uint_as_float(r.y << 16);
        v[3] = __uint_as_float(r.y & 0xffff0000u);
    }
    __device__ void set(const float (&v)[V])
    {
        const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]);
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2], v[3]);
        r.x = *reinterpret_cast<const unsigned *>(&a);
        r.y = *reinterpret_cast<const unsigned *>(&b);
    }
};

// exp(g).  Near 0 the decay is 1 + expm1(g) by its Taylor series (the next
// term, g^6 / 720, is below 2^-27 of 1 for |g| < 1/8): the last addition is
// the only rounding of the size of the result, and it has no preferred sign.
// expf's error, although below one unit in the last place, does, and a
// channel that remembers thousands of tokens adds it up once a token: 1.1e-5
// of the final state at 8192 tokens against 2e-6.  Larger |g| forget within a
// few tokens.
__device__ __forceinline__ float decay(float g)
{
    float p = fmaf(g, 1.f / 120.f, 1.f / 24.f);
    p = fmaf(g, p, 1.f / 6.f);
    p = fmaf(g, p, 0.5f);
    p = fmaf(g * g, p, g);
    return fabsf(g) < 0.125f ? 1.f + p : expf(g);
}

// ---- positions ------------------------------------------------------------

// The channels of a thread: V consecutive ones (VEC: one wide access each), or
// every LANES-th (any alignment).
template <bool VEC> __device__ __forceinline__ int local_channel(int lane, int v)
{
    return VEC ? lane * V + v : v * LANES + lane;
}

// One token tensor as a thread sees it: its channels' offsets in a row.
template <typename T, bool VEC> struct Col {
    T *p;
    int off[VEC ? 1 : V];   // elements after p
    __device__ Col(const void *base, int64_t sh, int64_t c0, int lane, int64_t C, int D)
    {
        int64_t first = 0;
#pragma unroll
        for (int v = 0; v < (VEC ? 1 : V); ++v) {
            int64_t c = c0 + local_channel<VEC>(lane, v);
            if (c >= C)
                c = c0;   // not accessed
            const int64_t o = c / D * sh + c % D;
            if (v == 0)
                first = o;
            off[v] = (int)(o - first);
        }
        p = const_cast<T *>(static_cast<const T *>(base)) + first;
    }
    __device__ T *row(int2 bt, int64_t sb, int64_t st) const { return p + bt.x * sb + bt.y * st; }
    // the row's values to the thread's slot: asynchronously where they are wide
    __device__ void fetch(const T *q, unsigned on, Four<T> *slot) const
    {
        if constexpr (VEC) {
            const unsigned to = (unsigned)__cvta_generic_to_shared(slot);
            if constexpr (sizeof(*slot) == 16)
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(q)
                             : "memory");
            else
                asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(q)
                             : "memory");
        } else {
            float f[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                f[v] = on >> v & 1 ? ldt(q + off[v]) : 0.f;
            slot->set(f);
        }
    }
    __device__ void store(T *q, unsigned on, const float (&f)[V]) const
    {
        if constexpr (VEC) {
            Four<T> r;
            r.set(f);
            *reinterpret_cast<decltype(r.r) *>(q) = r.r;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (on >> v & 1)
                    stt(q + off[v], f[v]);
        }
    }
};

// The tile's tokens: (batch row, token) and the number of the sequence.
struct Tokens {
    int2 at[SCAN_TILE];
    int seq[SCAN_TILE];
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
            *edge = p + (LAST ? (a.reverse ? t - lo : hi - 1 - t) : (a.reverse ? t - hi + 1 : lo - t));
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
    const unsigned ss = __ballot_sync(0xffffffffu, start), es = __ballot_sync(0xffffffffu, end);
    __syncwarp();
    const int shift = lane / LANES * L;
    return Marks{ss >> shift & ((1u << L) - 1), es >> shift & ((1u << L) - 1)};
}

// A state vector's values at the thread's channels (0 where absent).
template <bool VEC>
__device__ __forceinline__ void get_state(const float *from, int64_t n, int64_t C, int64_t c0,
                                          int lane, unsigned on, float (&s)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        s[v] = from && (on >> v & 1) ? from[n * C + c0 + local_channel<VEC>(lane, v)] : 0.f;
}
template <bool VEC>
__device__ __forceinline__ void put_state(float *to, int64_t n, int64_t C, int64_t c0, int lane,
                                          unsigned on, const float (&s)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        if (on >> v & 1)
            to[n * C + c0 + local_channel<VEC>(lane, v)] = s[v];
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

__device__ __forceinline__ unsigned long long pack(float A, float B)
{
    unsigned a = __float_as_uint(A);
    if (a == 0xffffffffu)   // a NaN that would read as EMPTY
        a = 0x7fffffffu;
    return (unsigned long long)a << 32 | __float_as_uint(B);
}
__device__ __forceinline__ void publish(unsigned long long *p, float A, float B)
{
    asm volatile("st.relaxed.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(pack(A, B)) : "memory");
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
    if (t - t0 <= WAIT_NS)
        return false;
    *flag = 0;
    atomicExch(&g_scan_error, LA_ERR_TIMEOUT);
    return true;
}

struct Shared {
    float A[WARPS][CT], B[WARPS][CT];     // the warps' maps, in processing order
    float fB[WARPS][CT];                  // backward: B of their forward maps (A is the same)
    float base[CT], pA[PARTS][CT], pB[PARTS][CT];
    int reset[WARPS], freset[WARPS];      // whether a sequence starts in the warp's tokens
    Tokens tk[2];                         // by stage, as the next three
    int64_t edge[2];                      // where the chain's sequence began (its position)
    int entered[2];                       // backward: the forward chain enters the tile
    unsigned item;                        // the one after the present one
};

// The map of a run of tokens; r: a sequence starts in it (what comes before is
// dropped, A is not used).
struct Map {
    float A, B;
    int r;
};
__device__ __forceinline__ float through(float A, float B, int r, float s)
{
    return r ? B : fmaf(A, s, B);
}
// A product of decays that are not zero stays above zero where fp32 underflows:
// an infinite state stays infinite, as it does token by token.
__device__ __forceinline__ float times(float a, float b)
{
    const float r = a * b;
    return r == 0.f && a != 0.f && b != 0.f ? 1.4e-45f : r;
}

// The state that enters tile m (tiles numbered in the order of the chain, ms
// the tile in which its sequence starts, ms < m), for channel threadIdx.x % CT
// of the tile, left in sm.base / pA / pB for entering() below.
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
__device__ __forceinline__ void tile_carry(const Link &k, Shared &sm, int64_t C, int64_t c0, int m,
                                           int ms)
{
    const int ch = threadIdx.x % CT, part = threadIdx.x / CT;
    const bool on = c0 + ch < C;
    const int gs = m / GROUP * GROUP;
    const bool far = ms < gs;
    const int first = far ? gs : ms + 1, each = (m - first + PARTS - 1) / PARTS;
    const int lo = first + part * each;
    const unsigned long long *ag = k.agg + c0 + ch + (int64_t)lo * C;
    const unsigned long long *bp = far ? k.inc + (int64_t)(m / GROUP - 1) * C + c0 + ch
                                       : k.agg + c0 + ch + (int64_t)ms * C;
    const int n = on ? min(each, m - lo) : 0;   // the thread's tiles
    const bool base = on && part == 0;
    unsigned long long v[EACH], b = base ? EMPTY : 0, t0 = 0;
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
    if (part == 0)
        sm.base[ch] = __uint_as_float((unsigned)b);
    sm.pA[part][ch] = A;
    sm.pB[part][ch] = B;
}
__device__ __forceinline__ float entering(const Shared &sm, int ch)
{
    float s = sm.base[ch];
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
        s = fmaf(sm.pA[q][ch], s, sm.pB[q][ch]);
    return s;
}

// The map of all WARPS' tokens (BACK: from the last to the first), channel ch.
template <bool BACK>
__device__ __forceinline__ Map tile_map(const float (&A)[WARPS][CT], const float (&B)[WARPS][CT],
                                        const int (&reset)[WARPS], int ch)
{
    Map m{1.f, 0.f, 0};
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
        const int w = BACK ? WARPS - 1 - i : i;
        m.B = through(A[w][ch], B[w][ch], reset[w], m.B);
        m.A = times(m.A, A[w][ch]);
        m.r |= reset[w];
    }
    return m;
}

// What a thread keeps of a tile whose copies it has issued.
struct Tile {
    unsigned item;
    int count;        // tokens of the thread's group
    unsigned on;      // bit v: channel v is there
    Marks mk;
};

// The slots of a stage: [token of the group][thread].
template <typename T> __device__ __forceinline__ Four<T> *slots(uint8_t *base)
{
    return reinterpret_cast<Four<T> *>(base) + threadIdx.x;
}
template <typename T> constexpr int slot_bytes() { return L * THREADS * (int)sizeof(Four<T>); }

// Looks the tile's tokens up and issues the copies of its tokens (BACK: do too).
template <bool BACK, typename T, typename TG, bool VEC>
__device__ __forceinline__ Tile issue(const ScanArgs &a, const Link &k, Shared &sm,
                                      uint8_t *stage, int st, unsigned item, int64_t C, int64_t P)
{
    const int lane = threadIdx.x % LANES, group = threadIdx.x / LANES, warp = threadIdx.x / 32;
    Tile t{item, 0, 0, Marks{0, 0}};
    if (item >= (unsigned)k.tiles * (unsigned)k.parts)
        return t;
    const int m = (int)(item / (unsigned)k.parts), tile = BACK ? k.tiles - 1 - m : m;
    const int64_t c0 = (int64_t)(item % (unsigned)k.parts) * CT, p0 = (int64_t)tile * SCAN_TILE;
#pragma unroll
    for (int v = 0; v < V; ++v)
        t.on |= (c0 + local_channel<VEC>(lane, v) < C ? 1u : 0u) << v;
    t.count = t.on ? (int)max((int64_t)0, min((int64_t)L, P - p0 - group * L)) : 0;
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
    const Col<T, VEC> x(a.x.p, a.x.sh, c0, lane, C, a.D);
    const Col<TG, VEC> g(a.g.p, a.g.sh, c0, lane, C, a.D);
    const Col<T, VEC> d(BACK ? a.d_o.p : a.x.p, BACK ? a.d_o.sh : a.x.sh, c0, lane, C, a.D);
    Four<T> *xs = slots<T>(stage), *ds = slots<T>(stage + slot_bytes<T>() + slot_bytes<TG>());
    Four<TG> *gs = slots<TG>(stage + slot_bytes<T>());
#pragma unroll
    for (int e = 0; e < L; ++e) {
        if (e < t.count) {
            const int2 bt = sm.tk[st].at[group * L + e];
            x.fetch(x.row(bt, a.x.sb, a.x.st), t.on, xs + e * THREADS);
            g.fetch(g.row(bt, a.g.sb, a.g.st), t.on, gs + e * THREADS);
            if (BACK)
                d.fetch(d.row(bt, a.d_o.sb, a.d_o.st), t.on, ds + e * THREADS);
        }
    }
    return t;
}

template <bool BACK, typename T, typename TG> constexpr int stage_bytes()
{
    return slot_bytes<T>() * (BACK ? 2 : 1) + slot_bytes<TG>();
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
    // items are taken in the order of the chain, so that whatever a tile waits
    // for is held by a CTA that runs and has nothing before it to wait for
    if (threadIdx.x == 0)
        sm.item = k.head ? atomicAdd(k.head, 1u) + 1u : blockIdx.x;
    __syncthreads();
    Tile cur = issue<false, T, TG, VEC>(a, k, sm, ring, 0, sm.item, C, P);
    copies_issued();
    __syncthreads();
    if (threadIdx.x == 0)
        sm.item = k.head ? atomicAdd(k.head, 1u) + 1u : items;
    for (int st = 0;; st ^= 1) {
        if (cur.item >= items)
            break;
        __syncthreads();
        const Tile nxt = issue<false, T, TG, VEC>(a, k, sm, ring + (st ^ 1) * STAGE, st ^ 1,
                                                  sm.item, C, P);
        copies_issued();
        unsigned after = items;
        if (threadIdx.x == 0 && k.head && nxt.item < items)
            after = atomicAdd(k.head, 1u) + 1u;
        copies_before_last();
        const Tokens &tk = sm.tk[st];
        const Four<T> *xs = slots<T>(ring + st * STAGE);
        const Four<TG> *gs = slots<TG>(ring + st * STAGE + slot_bytes<T>());
        const int tile = (int)(cur.item / (unsigned)k.parts);
        const int64_t c0 = (int64_t)(cur.item % (unsigned)k.parts) * CT;
        const int64_t p0 = (int64_t)tile * SCAN_TILE;
        const unsigned starts = cur.mk.starts;
        // the thread's tokens composed to s -> A s + B; their decays are kept
        float d[L][V], A[V], B[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            A[v] = 1.f, B[v] = 0.f;
#pragma unroll
        for (int e = 0; e < L; ++e) {
            if (e < cur.count) {
                if (starts >> e & 1)   // from here on A is not used
                    get_state<VEC>(a.init, tk.seq[slot + e], C, c0, lane, cur.on, B);
                float xv[V], gv[V];
                xs[e * THREADS].get(xv);
                gs[e * THREADS].get(gv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    d[e][v] = decay(gv[v]);
                    B[v] = fmaf(d[e][v], B[v], xv[v]);
                    A[v] *= d[e][v];
                }
            }
        }
        // the two groups of a warp, then the warps
        const int r = starts != 0;
        float eA[V], eB[V];   // the even group's map, for the odd group
        const int er = __shfl_up_sync(0xffffffffu, r, LANES);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            eA[v] = __shfl_up_sync(0xffffffffu, A[v], LANES);
            eB[v] = __shfl_up_sync(0xffffffffu, B[v], LANES);
        }
        if (odd) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int ch = local_channel<VEC>(lane, v);
                sm.A[warp][ch] = times(A[v], eA[v]);
                sm.B[warp][ch] = through(A[v], B[v], r, eB[v]);
            }
            if (lane == 0)
                sm.reset[warp] = r | er;
        }
        __syncthreads();
        const int64_t edge = sm.edge[st];
        const bool chained = p0 > edge;   // the tile goes on with an earlier one's state
        const int64_t ch = c0 + threadIdx.x;
        const bool speaks = threadIdx.x < CT && ch < C && k.head;
        Map whole{1.f, 0.f, 0};
        if (speaks) {
            whole = tile_map<false>(sm.A, sm.B, sm.reset, threadIdx.x);
            if (!(k.withhold && tile == 0))
                publish(k.agg + tile * C + ch, whole.A, whole.B);
        }
        float s[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            s[v] = 0.f;
        if (chained) {
            tile_carry(k, sm, C, c0, tile, (int)(edge / SCAN_TILE));
            __syncthreads();
            if (speaks) {
                const float in = entering(sm, threadIdx.x);
                if (tile % GROUP == GROUP - 1)
                    publish(k.inc + tile / GROUP * C + ch, 0.f,
                            through(whole.A, whole.B, whole.r, in));
                if (a.states)
                    a.states[tile * C + ch] = in;
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                s[v] = entering(sm, local_channel<VEC>(lane, v));
        } else if (speaks && tile % GROUP == GROUP - 1) {
            publish(k.inc + tile / GROUP * C + ch, 0.f, whole.B);
        }
        // the state that enters the thread's tokens
        for (int w = 0; w < warp; ++w) {
            const int rw = sm.reset[w];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = local_channel<VEC>(lane, v);
                s[v] = through(sm.A[w][c], sm.B[w][c], rw, s[v]);
            }
        }
        if (odd) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                s[v] = through(eA[v], eB[v], er, s[v]);
        }
        if (a.o.p || a.fin) {
            const Col<T, VEC> o(a.o.p, a.o.sh, c0, lane, C, a.D);
#pragma unroll
            for (int e = 0; e < L; ++e) {
                if (e < cur.count) {
                    if (starts >> e & 1)
                        get_state<VEC>(a.init, tk.seq[slot + e], C, c0, lane, cur.on, s);
                    float xv[V];
                    xs[e * THREADS].get(xv);
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        s[v] = fmaf(d[e][v], s[v], xv[v]);
                    if (a.o.p)
                        o.store(o.row(tk.at[slot + e], a.o.sb, a.o.st), cur.on, s);
                    if (a.fin && (cur.mk.ends >> e & 1))
                        put_state<VEC>(a.fin, tk.seq[slot + e], C, c0, lane, cur.on, s);
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
        sm.item = k.head ? atomicAdd(k.head, 1u) + 1u : blockIdx.x;
    __syncthreads();
    Tile cur = issue<true, T, TG, VEC>(a, k, sm, ring, 0, sm.item, C, P);
    copies_issued();
    __syncthreads();
    if (threadIdx.x == 0)
        sm.item = k.head ? atomicAdd(k.head, 1u) + 1u : items;
    for (int st = 0;; st ^= 1) {
        if (cur.item >= items)
            break;
        __syncthreads();
        const Tile nxt = issue<true, T, TG, VEC>(a, k, sm, ring + (st ^ 1) * STAGE, st ^ 1,
                                                 sm.item, C, P);
        copies_issued();
        unsigned after = items;
        if (threadIdx.x == 0 && k.head && nxt.item < items)
            after = atomicAdd(k.head, 1u) + 1u;
        copies_before_last();
        const Tokens &tk = sm.tk[st];
        const Four<T> *xs = slots<T>(ring + st * STAGE);
        const Four<TG> *gs = slots<TG>(ring + st * STAGE + slot_bytes<T>());
        const Four<T> *ds = slots<T>(ring + st * STAGE + slot_bytes<T>() + slot_bytes<TG>());
        const int m = (int)(cur.item / (unsigned)k.parts), tile = k.tiles - 1 - m;
        const int64_t c0 = (int64_t)(cur.item % (unsigned)k.parts) * CT;
        const int64_t pe = min(P, (int64_t)(tile + 1) * SCAN_TILE) - 1;   // the last position
        const Marks mk = cur.mk;
        // the thread's map of the forward chain and of the backward chain
        float d[L][V];
        float fA[V], fB[V], A[V], B[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            fA[v] = A[v] = 1.f, fB[v] = B[v] = 0.f;
#pragma unroll
        for (int e = 0; e < L; ++e) {
            if (e < cur.count) {
                if (mk.starts >> e & 1)
                    get_state<VEC>(a.init, tk.seq[slot + e], C, c0, lane, cur.on, fB);
                float gv[V], xv[V];
                gs[e * THREADS].get(gv);
                xs[e * THREADS].get(xv);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    d[e][v] = decay(gv[v]);
                    fB[v] = fmaf(d[e][v], fB[v], xv[v]);
                    fA[v] *= d[e][v];
                }
            }
        }
#pragma unroll
        for (int e = L - 1; e >= 0; --e) {
            if (e < cur.count) {
                if (mk.ends >> e & 1)
                    get_state<VEC>(a.dfin, tk.seq[slot + e], C, c0, lane, cur.on, B);
                float dv[V];
                ds[e * THREADS].get(dv);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    B[v] = d[e][v] * (dv[v] + B[v]);
            }
        }
        // the same decays: one product serves both chains
#pragma unroll
        for (int v = 0; v < V; ++v)
            A[v] = fA[v];
        // each group's neighbour: the even group's forward map for the odd one,
        // the odd group's backward map for the even one
        const int fr = mk.starts != 0, r = mk.ends != 0;
        float oA[V], oB[V];
        const int orr = __shfl_xor_sync(0xffffffffu, odd ? r : fr, LANES);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            oA[v] = __shfl_xor_sync(0xffffffffu, fA[v], LANES);
            oB[v] = __shfl_xor_sync(0xffffffffu, odd ? B[v] : fB[v], LANES);
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int c = local_channel<VEC>(lane, v);
            if (odd) {
                sm.fB[warp][c] = through(fA[v], fB[v], fr, oB[v]);
            } else {
                sm.A[warp][c] = times(A[v], oA[v]);
                sm.B[warp][c] = through(A[v], B[v], r, oB[v]);
            }
        }
        if (lane == 0) {
            if (odd)
                sm.freset[warp] = fr | orr;
            else
                sm.reset[warp] = r | orr;
        }
        __syncthreads();
        const int64_t edge = sm.edge[st];
        const int64_t ch = c0 + threadIdx.x;
        const bool speaks = threadIdx.x < CT && ch < C && k.head;
        Map whole{1.f, 0.f, 0};
        if (speaks) {
            whole = tile_map<true>(sm.A, sm.B, sm.reset, threadIdx.x);
            if (!(k.withhold && m == 0))
                publish(k.agg + m * C + ch, whole.A, whole.B);
        }
        // the states before the thread's tokens
        float x[L][V];
        {
            float s[V];
            get_state<VEC>(sm.entered[st] ? a.states : nullptr, tile, C, c0, lane, cur.on, s);
            for (int w = 0; w < warp; ++w) {
                const int rw = sm.freset[w];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const int c = local_channel<VEC>(lane, v);
                    s[v] = through(sm.A[w][c], sm.fB[w][c], rw, s[v]);
                }
            }
            if (odd) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    s[v] = through(oA[v], oB[v], orr, s[v]);
            }
#pragma unroll
            for (int e = 0; e < L; ++e) {
                if (e < cur.count) {
                    if (mk.starts >> e & 1)
                        get_state<VEC>(a.init, tk.seq[slot + e], C, c0, lane, cur.on, s);
                    float xv[V];
                    xs[e * THREADS].get(xv);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        x[e][v] = s[v];
                        s[v] = fmaf(d[e][v], s[v], xv[v]);
                    }
                }
            }
        }
        float K[V];
#pragma unroll
        for (int v = 0; v < V; ++v)
            K[v] = 0.f;
        if (pe < edge) {   // a later tile's gradient enters
            tile_carry(k, sm, C, c0, m, k.tiles - 1 - (int)(edge / SCAN_TILE));
            __syncthreads();
            if (speaks && m % GROUP == GROUP - 1)
                publish(k.inc + m / GROUP * C + ch, 0.f,
                        through(whole.A, whole.B, whole.r, entering(sm, threadIdx.x)));
#pragma unroll
            for (int v = 0; v < V; ++v)
                K[v] = entering(sm, local_channel<VEC>(lane, v));
        } else if (speaks && m % GROUP == GROUP - 1) {
            publish(k.inc + m / GROUP * C + ch, 0.f, whole.B);
        }
        for (int w = WARPS - 1; w > warp; --w) {
            const int rw = sm.reset[w];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = local_channel<VEC>(lane, v);
                K[v] = through(sm.A[w][c], sm.B[w][c], rw, K[v]);
            }
        }
        if (!odd) {
#pragma unroll
            for (int v = 0; v < V; ++v)
                K[v] = through(oA[v], oB[v], orr, K[v]);
        }
        {
            const Col<T, VEC> dx(a.dx.p, a.dx.sh, c0, lane, C, a.D);
            const Col<TG, VEC> dg(a.dg.p, a.dg.sh, c0, lane, C, a.D);
#pragma unroll
            for (int e = L - 1; e >= 0; --e) {
                if (e < cur.count) {
                    if (mk.ends >> e & 1)
                        get_state<VEC>(a.dfin, tk.seq[slot + e], C, c0, lane, cur.on, K);
                    float G[V], y[V];
                    ds[e * THREADS].get(G);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        G[v] += K[v];
                        K[v] = d[e][v] * G[v];
                        y[v] = K[v] * x[e][v];
                    }
                    const int2 bt = tk.at[slot + e];
                    dx.store(dx.row(bt, a.dx.sb, a.dx.st), cur.on, G);
                    dg.store(dg.row(bt, a.dg.sb, a.dg.st), cur.on, y);
                    if (a.dinit && (mk.starts >> e & 1))
                        put_state<VEC>(a.dinit, tk.seq[slot + e], C, c0, lane, cur.on, K);
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
