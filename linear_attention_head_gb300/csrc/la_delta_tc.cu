// la_delta_tc.cu -- the gated delta rule in chunks of 64 tokens on the tensor
// cores (tcgen05, TMA, TMEM): bf16, D and E multiples of 8 up to 128.
//
// Per sequence and value head, S (D x E) entering a chunk, G the running sums of
// g in it, M_ij = exp(G_i - G_j) for j <= i, token i's write beta_i k_i e_i^T:
//
//     A = strictly lower part of M * (K K^T),   (I + A beta) B = A
//     X = V - e^G K S,                          Eps = X - B (beta X)
//     O = scale e^G Q S + P (beta Eps),         P = scale M * (Q K^T)
//     S' = e^G_C S + K^T (kappa beta Eps),      kappa_j = exp(G_C - G_j)
//
// and back, K' = dL/dS' (called G below where no confusion arises):
//
//     W = P^T dO + kappa K K',                  R = W - B^T (beta W)
//     dV = beta R,  dbeta_i = R_i . Eps_i
//     dL/dS = e^G_C K' + (scale e^G Q)^T dO - (e^G K)^T dV
//     dQ = scale e^G dO S^T + W1 K,             W1 = scale M * (dO Eps^T) beta
//     dK = -e^G dV S^T + W2 K                   (row: as the one that reads S)
//        + W1^T Q + W2^T K + kappa beta Eps K'^T    (col: as the one that writes)
//        with W2 = -M * (dV Eps^T) beta, strictly lower
//     dg_t = sum over i >= t in the chunk of (q_i.dq_i + k_i.(row_i - col_i)) + <S', K'>.
//
// B needs neither S nor a division by beta.  Four kernels:
//   delta_prep     B of every chunk, all chunks in parallel (fp32 diagonal blocks, mma.sync
//                  between)
//   delta_sweep    <false>: the forward, a CTA a (sequence, head), chunk by chunk
//                  <true>: the backward's K' and dV, from the last chunk to the first
//   delta_grads    dQ, dK, dg, dbeta, all chunks in parallel
// and where (sequence, head) pairs are few, long sequences in segments that run at
// once: S' = Phi S + H over a segment, Phi (D x D) and H by sweeps without outputs that
// start from the identity without values and from zero, then a scan over the segments
// (delta_scan) and the sweeps proper from the states that it gives.  Back the same with
// Phi^T, which the forward's sweeps have left.
//
// The sweeps work transposed: the 128 TMEM lanes are the value channels, the
// columns tokens or key channels.  So S^T, X^T, Eps^T come out of one product and
// go into the next as its A operand through TMEM, and K, Q, B are B operands as
// they lie.  A chunk is a chain: K S -> X -> B (beta X) -> Eps -> K^T Eps -> S.
// Chunks of 64: B costs a quarter of what 128 would, and half the bytes a token.
//
// Precision: inputs are exact in bf16; every other operand of the chain (S, X,
// Eps, B, P) is held as two bf16, hi + lo, 16 bits of it, and multiplied
// hi hi + hi lo + lo hi with fp32 sums: the states stay within 2^-17 a factor
// instead of 2^-9.  The tensor cores have room: the chain's latency is what a
// chunk takes.  delta_grads rounds its operands (S, K', Eps, R, W1, W2) to bf16
// once: its outputs are bf16 gradients that no later chunk depends on.  dV leaves the
// sweep, which has R in fp32.  The gates' running sums are two floats each.
//
// On one GB300, b4 h32 n8192 d128, forward and backward 1.80 ms: delta_prep 0.21, the
// sweeps 0.51 and 0.55 (DRAM busy 46% and 41%, the tensor pipe 25% and 21%: the chain's
// latency, 4 us a chunk), delta_grads 0.52 (3.0 GB, 0.85 of the copy rate).  With 16
// query and key heads for the 32 value heads it is 2.80: delta_grads 0.73, which writes
// fp32 parts of dq and dk a value head, and 0.40 for each of their sums over a group.

#include <climits>

#include "la_f32x2.cuh"
#include "la_tc_common.cuh"

namespace la {
namespace {

constexpr int C = 64;                           // tokens a chunk
constexpr int BTILE = 16384;                    // B hi, B lo: [64][64] bf16 each
constexpr int STILE = 32768;                    // S^T or K'^T: [2][128 e][64 d] bf16
constexpr int ETILE = 16384;                    // Eps or R: [2][64 tokens][64 e] bf16
// per token: -e^G, -beta, kappa, kappa beta, -e^G beta, beta, G / ln 2 as two floats,
// each for a chunk's 64 tokens in a row
constexpr int TNEG = 0, TNB = 1, TKAP = 2, TKB = 3, TNGB = 4, TBETA = 5, TLOG = 6, TLOW = 7,
              TABS = 8;
constexpr int TAB = TABS * C * 4;
constexpr float LEAST_GATE = -100.f;            // e^-100 is 0 beside anything kept

// Where a chunk lies.  Chunk slots: ceil(T / 64) a dense row; cu[n] / 64 + n on
// packed, which leaves every sequence room for its ceil(len / 64).
__host__ __device__ inline int64_t slots_of(int N, int T, bool packed)
{
    return packed ? (int64_t)T / C + N : (int64_t)N * ((T + C - 1) / C);
}
struct Seq {
    int n;
    int64_t row, bos, len, slot;        // slot: of the sequence's first chunk
};
__device__ __forceinline__ Seq sequence(const int32_t *cu, int T, int n)
{
    Seq q;
    q.n = n;
    if (cu) {
        q.row = 0;
        q.bos = cu[n];
        q.len = (int64_t)cu[n + 1] - q.bos;
        q.slot = q.bos / C + n;
    } else {
        q.row = n;
        q.bos = 0;
        q.len = T;
        q.slot = (int64_t)n * ((T + C - 1) / C);
    }
    return q;
}
// The sequence that slot belongs to (the last one whose first slot is not above).
__device__ __forceinline__ Seq sequence_of_slot(const int32_t *cu, int T, int N, int64_t slot)
{
    if (!cu)    // slots of all heads together are below 2^31
        return sequence(nullptr, T, (int)slot / ((T + C - 1) / C));
    int lo = 0, hi = N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (cu[mid] / C + mid <= slot)
            lo = mid;
        else
            hi = mid - 1;
    }
    return sequence(cu, T, lo);
}

struct Scratch {
    uint8_t *b;         // [slot][H] BTILE
    float *tab;         // [slot][H][TABS][64]
    uint8_t *s, *e;     // [slot][H] STILE, ETILE (kept for the backward; or null)
    uint8_t *k, *r;     // backward: [slot][H] STILE, ETILE
    // segments: [N segs][H][D][D], and [N segs][H][D][E] each: Phi, H, entering states
    float *phi, *own, *enter;
    float *dqp, *dkp;   // backward, shared heads: [B][T][H][D] fp32
};

__device__ __forceinline__ float gate_at(const Tok &g, int bf16, int64_t row, int64_t t, int h)
{
    const int64_t at = row * g.sb + t * g.st + (int64_t)h * g.sh;
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(g.p)[at])
                : static_cast<const float *>(g.p)[at];
}

// bwait in few instructions, the clock read only every 16th time: a chunk is a dozen
// hand-offs one after another, and a kernel that outgrows the instruction cache waits
// for its code (0.19 MB of it: 0.62 ms a sweep at b4 h32 n8192)
__device__ __forceinline__ bool wait_for(uint64_t *bar, uint32_t parity, volatile int *abort_flag)
{
    uint64_t t0 = 0;
#pragma unroll 1
    for (int i = 1;; ++i) {
        if (mbar_try_wait(bar, parity))
            return true;
        if (i & 15)
            continue;
        if (*abort_flag)
            return false;
        const uint64_t now = globaltimer_ns();
        if (t0 == 0)
            t0 = now;
        if (now - t0 > TC_WAIT_NS) {
            *abort_flag = 1;
            atomicExch(&g_tc_error, TC_ERR_TIMEOUT);
            return false;
        }
    }
}

// Without a clock: for the chain's and the side warps, which wait for what the other
// warps do or give up.  Those raise abort_flag when a wait of theirs runs out, the last
// products' too, and otherwise end only with everything done that is waited for here.
__device__ __forceinline__ bool wait_here(uint64_t *bar, uint32_t parity, volatile int *abort_flag)
{
    int i = 0;
#pragma unroll 1
    while (!mbar_try_wait(bar, parity))
        if ((++i & 15) == 0 && *abort_flag)     // seldom: it is shared memory's time too
            return false;
    return true;
}
// (The backward's sweep was slower with it, 45 us to 67 at b2 h8 n2047 d64.)
template <bool BWD>
__device__ __forceinline__ bool wait_role(uint64_t *bar, uint32_t parity, volatile int *abort_flag)
{
    return BWD ? wait_for(bar, parity, abort_flag) : wait_here(bar, parity, abort_flag);
}
// the same as a call: for the warps that hold little in registers
__device__ __noinline__ bool wait_call(uint64_t *bar, uint32_t parity, volatile int *abort_flag)
{
    return wait_for(bar, parity, abort_flag);
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b)
{
    return un(la::mul2(f2(a.x, a.y), f2(b.x, b.y)));
}
__device__ __forceinline__ float2 add2(float2 a, float2 b)
{
    return un(la::add2(f2(a.x, a.y), f2(b.x, b.y)));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c)
{
    return un(la::fma2(f2(a.x, a.y), f2(b.x, b.y), f2(c.x, c.y)));
}
// One lane of a whole warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "elect.sync _|p, 0xffffffff;\n\t"
                 "selp.u32 %0, 1, 0, p;\n\t}"
                 : "=r"(one));
    return one != 0;
}
// x as hi + lo, each two bf16.
__device__ __forceinline__ void split2(float2 x, uint32_t &hi, uint32_t &lo)
{
    hi = pack_bf16x2(x.x, x.y);
    const float2 rest = fma2(make_float2(bf16lo(hi), bf16hi(hi)), make_float2(-1.f, -1.f), x);
    lo = pack_bf16x2(rest.x, rest.y);
}
__device__ __forceinline__ float2 pair_of(const uint32_t (&r)[32], int m)
{
    return make_float2(__uint_as_float(r[2 * m]), __uint_as_float(r[2 * m + 1]));
}
__device__ __forceinline__ void put_pair(uint32_t (&r)[32], int m, float2 x)
{
    r[2 * m] = __float_as_uint(x.x);
    r[2 * m + 1] = __float_as_uint(x.y);
}
// 2^x, within 2^-22 of it
__device__ __forceinline__ float exp2_fast(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Running sums of gates as two floats (hi, lo; 2^-46 or so): strong gates leave sums of
// thousands, and the decays between slow ones after them are differences of such sums.
// In one float a decay was off by up to 2.4e-4 (32 resets in a chunk), so now by 2^-24 a
// unit of the difference itself.
__device__ __forceinline__ float2 sum_two(float2 a, float2 b)
{
    const float s = a.x + b.x, t = s - a.x;
    const float e = (a.x - (s - t)) + (b.x - t) + (a.y + b.y);
    const float hi = s + e;
    return make_float2(hi, e - (hi - s));
}
__device__ __forceinline__ float less_two(float2 a, float2 b) { return (a.x - b.x) + (a.y - b.y); }
// times log2 e
__device__ __forceinline__ float2 to_log2(float2 a)
{
    constexpr float H = 1.4426950408889634f, LO = (float)(1.4426950408889634 - (double)H);
    const float p = a.x * H;
    const float e = fmaf(a.x, LO, fmaf(a.y, H, fmaf(a.x, H, -p)));
    const float hi = p + e;
    return make_float2(hi, e - (hi - p));
}

__device__ __forceinline__ void bulk_prefetch(const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_store(void *dst, const void *src, uint32_t bytes)
{
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                 "r"(smem_u32(src)), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
                 " [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// ---- B of every chunk -----------------------------------------------------------
//
// K K^T by mma.sync (bf16 exact, fp32 sums), then the triangular system: diagonal
// blocks of 16 by substitution in fp32, a thread a column, and blocks joined
// 16 -> 32 -> 64 on the tensor cores,
//     M = A21 - A21 (beta B11),   B21 = M - B22 (beta M),
// the factors as hi + lo (hi hi, hi lo, lo hi), A21 and M in the fp32 fragments that
// K K^T left in registers.  The left factors (A21, then B) end as B itself, hi and lo:
// what is written out.  (The joins by fp32 FMAs read their factors again and again from
// shared memory: 0.30 ms for the 16384 chunks of b4 h32 n8192, then 0.22, now 0.21.)

constexpr int PREP = 128;
constexpr int KP = 136;         // bf16 a row of K in shared memory
constexpr int LP = 72;          // bf16 a row of the factors: eight rows, eight banks of 16 bytes
constexpr int DP = 20;          // floats a row of the diagonal blocks

__device__ __forceinline__ void ldm_x4(uint32_t (&r)[4], const void *p)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p))
                 : "memory");
}
__device__ __forceinline__ void ldm_x4_trans(uint32_t (&r)[4], const void *p)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(smem_u32(p))
                 : "memory");
}
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3},"
                 " {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

typedef __nv_bfloat16 Factor[2][C][LP];         // hi, lo

// acc (16 rows from r0, 8 N columns from c0) -= left[r0 ..][k0 .. k0 + K) right[k0 ..][c0 ..]
template <int K, int N>
__device__ __forceinline__ void minus_product(float (*acc)[4], const Factor &left,
                                              const Factor &right, int r0, int k0, int c0)
{
    const int lane = threadIdx.x & 31, r = lane & 15, half = 8 * (lane >> 4);
    float sum[N][4] = {};
#pragma unroll
    for (int kk = 0; kk < K; kk += 16) {
        uint32_t l[2][4];
        ldm_x4(l[0], &left[0][r0 + r][k0 + kk + half]);
        ldm_x4(l[1], &left[1][r0 + r][k0 + kk + half]);
#pragma unroll
        for (int n = 0; n < N; n += 2) {
            uint32_t x[2][4];
            ldm_x4_trans(x[0], &right[0][k0 + kk + r][c0 + 8 * n + half]);
            ldm_x4_trans(x[1], &right[1][k0 + kk + r][c0 + 8 * n + half]);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                mma_16816(sum[n + y], l[0], x[0][2 * y], x[0][2 * y + 1]);
                mma_16816(sum[n + y], l[1], x[0][2 * y], x[0][2 * y + 1]);
                mma_16816(sum[n + y], l[0], x[1][2 * y], x[1][2 * y + 1]);
            }
        }
    }
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
        for (int v = 0; v < 4; ++v)
            acc[n][v] -= sum[n][v];
}
// the fragments of 16 rows from r0, 8 N columns from c0, times f[row] (null: 1), as hi + lo
template <int N>
__device__ __forceinline__ void put_factor(Factor &to, const float (*acc)[4], int r0, int c0,
                                           const float *f)
{
    const int lane = threadIdx.x & 31, r = r0 + (lane >> 2), c = c0 + 2 * (lane & 3);
#pragma unroll
    for (int v = 0; v < 4; v += 2) {
        const float s = f ? f[r + 4 * v] : 1.f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
            uint32_t hi, lo;
            split2(make_float2(s * acc[n][v], s * acc[n][v + 1]), hi, lo);
            *reinterpret_cast<uint32_t *>(&to[0][r + 4 * v][c + 8 * n]) = hi;
            *reinterpret_cast<uint32_t *>(&to[1][r + 4 * v][c + 8 * n]) = lo;
        }
    }
}

__global__ void __launch_bounds__(PREP) delta_prep_kernel(const DeltaArgs a, const Scratch sc)
{
    // K, then the right factors: beta B of the first blocks, beta M of the second ones
    __shared__ __align__(16) uint8_t over[sizeof(Factor)];
    static_assert(sizeof(Factor) >= C * KP * sizeof(__nv_bfloat16), "the right factors lie over K");
    __nv_bfloat16 (*ks)[KP] = reinterpret_cast<__nv_bfloat16 (*)[KP]>(over);
    Factor &R = *reinterpret_cast<Factor *>(over);
    __shared__ __align__(16) Factor L;
    __shared__ __align__(16) float diag[4][16][DP];
    __shared__ float2 G[C], part[2];
    __shared__ float beta[C];
    const int64_t slot = (int)blockIdx.x / a.H;
    const int h = (int)blockIdx.x - (int)slot * a.H;
    const Seq q = sequence_of_slot(a.cu, a.T, a.N, slot);
    const int64_t t0 = (slot - q.slot) * C;
    if (t0 >= q.len)
        return;
    const int n = (int)min((int64_t)C, q.len - t0);     // tokens of this chunk
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t tile = slot * a.H + h;

    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k.p) + q.row * a.k.sb +
                             (q.bos + t0) * a.k.st + (int64_t)(h / a.k.hdiv) * a.k.sh;
    const int ksteps = (a.D + 15) / 16;
    float2 g = make_float2(0.f, 0.f);
    float b = 0.f;
    if (tid < n) {
        g.x = gate_at(a.g, a.gate_bf16, q.row, q.bos + t0 + tid, h);
        g.x = g.x < LEAST_GATE ? LEAST_GATE : g.x;      // (a NaN stays one)
        b = gate_at(a.beta, a.gate_bf16, q.row, q.bos + t0 + tid, h);
    }
    {   // every load on its way before the first is waited for
        uint4 v[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int i = (tid >> 4) + 8 * x, c = tid & 15;
            v[x] = make_uint4(0, 0, 0, 0);
            if (i < n && 8 * c < a.D)
                v[x] = *reinterpret_cast<const uint4 *>(k + i * a.k.st + 8 * c);
        }
#pragma unroll
        for (int x = 0; x < 8; ++x)
            *reinterpret_cast<uint4 *>(&ks[(tid >> 4) + 8 * x][8 * (tid & 15)]) = v[x];
    }
    if (tid < C) {
#pragma unroll
        for (int m = 1; m < 32; m *= 2) {
            const float2 y = make_float2(__shfl_up_sync(0xffffffffu, g.x, m),
                                         __shfl_up_sync(0xffffffffu, g.y, m));
            if (lane >= m)
                g = sum_two(g, y);
        }
        if (lane == 31)
            part[warp] = g;
        beta[tid] = b;
    }
    __syncthreads();
    if (tid < C) {
        g = tid < 32 ? g : sum_two(g, part[0]);
        float *tab = sc.tab + tile * TABS * C + tid;
        const float eg = expf(g.x), kap = expf(less_two(sum_two(part[1], part[0]), g));
        tab[TNEG * C] = -eg;
        tab[TNB * C] = -b;
        tab[TKAP * C] = kap;
        tab[TKB * C] = kap * b;
        tab[TNGB * C] = -eg * b;
        tab[TBETA * C] = b;
        g = to_log2(g);
        tab[TLOG * C] = g.x;
        tab[TLOW * C] = g.y;
        G[tid] = g;
    }
    // rows 16 warp .. of K K^T, columns up to the diagonal block
    float acc[8][4] = {};
    {
        const int r = lane & 15, half = lane >> 4;
        for (int kk = 0; kk < ksteps; ++kk) {
            uint32_t x[4];
            ldm_x4(x, &ks[16 * warp + r][16 * kk + 8 * half]);
#pragma unroll
            for (int jb = 0; jb < 4; ++jb)
                if (jb <= warp) {
                    uint32_t y[4];      // columns 16 jb: 0, 2 its first eight, 1, 3 the others
                    ldm_x4(y, &ks[16 * jb + r][16 * kk + 8 * half]);
                    mma_16816(acc[2 * jb], x, y[0], y[2]);
                    mma_16816(acc[2 * jb + 1], x, y[1], y[3]);
                }
        }
    }
    __syncthreads();    // K has been read, G written
    {   // A in place of K K^T; zeros from the diagonal on
        const int i0 = 16 * warp + (lane >> 2), j0 = 2 * (lane & 3);
        const float2 g0 = G[i0], g1 = G[i0 + 8];
#pragma unroll
        for (int nb = 0; nb < 8; ++nb)
            if (nb < 2 * (warp + 1)) {
                const int j = 8 * nb + j0;
                const float2 h0 = G[j], h1 = G[j + 1];
                acc[nb][0] = j < i0 ? exp2_fast(less_two(g0, h0)) * acc[nb][0] : 0.f;
                acc[nb][1] = j + 1 < i0 ? exp2_fast(less_two(g0, h1)) * acc[nb][1] : 0.f;
                acc[nb][2] = j < i0 + 8 ? exp2_fast(less_two(g1, h0)) * acc[nb][2] : 0.f;
                acc[nb][3] = j + 1 < i0 + 8 ? exp2_fast(less_two(g1, h1)) * acc[nb][3] : 0.f;
            }
        put_factor<8>(L, acc, 16 * warp, 0, nullptr);
#pragma unroll
        for (int jb = 0; jb < 4; ++jb)
            if (jb == warp)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int v = 0; v < 4; v += 2)
                        *reinterpret_cast<float2 *>(
                            &diag[warp][(lane >> 2) + 4 * v][8 * x + j0]) =
                            make_float2(acc[2 * jb + x][v], acc[2 * jb + x][v + 1]);
    }
    __syncwarp();
    // diagonal blocks of 16: column lane of block warp; L takes B, R beta B
    {
        const int b0 = 16 * warp, c = lane & 15;
        float z[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            float x = diag[warp][i][c];
#pragma unroll
            for (int m4 = 0; m4 < i; m4 += 4) {
                const float4 l = *reinterpret_cast<const float4 *>(&diag[warp][i][m4]);
                x = fmaf(-l.x, z[m4], x);
                if (m4 + 1 < i)
                    x = fmaf(-l.y, z[m4 + 1], x);
                if (m4 + 2 < i)
                    x = fmaf(-l.z, z[m4 + 2], x);
                if (m4 + 3 < i)
                    x = fmaf(-l.w, z[m4 + 3], x);
            }
            z[i] = beta[b0 + i] * x;
            // lanes 0-15 write hi, 16-31 lo; block 0's upper right in R is zero
            const __nv_bfloat16 xh = __float2bfloat16_rn(x), zh = __float2bfloat16_rn(z[i]);
            const bool low = lane >= 16;
            L[low][b0 + i][b0 + c] =
                low ? __float2bfloat16_rn(x - __bfloat162float(xh)) : xh;
            if (warp < 3)
                R[low][b0 + i][b0 + c] =
                    low ? __float2bfloat16_rn(z[i] - __bfloat162float(zh)) : zh;
            if (warp == 0)
                R[low][i][16 + c] = __float2bfloat16_rn(0.f);
        }
    }
    __syncthreads();
    if (warp & 1) {     // 16 -> 32: this warp's rows, the 16 columns before its diagonal block
        const int r0 = 16 * warp, c0 = r0 - 16;
        float m[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                m[x][v] = warp == 1 ? acc[x][v] : acc[4 + x][v];
        minus_product<16, 2>(m, L, R, r0, c0, c0);
        put_factor<2>(R, m, r0, c0, beta);
        __syncwarp();
        minus_product<16, 2>(m, L, R, r0, r0, c0);
        put_factor<2>(L, m, r0, c0, nullptr);
        __syncwarp();
        if (warp == 1)  // beta B in place of beta M
            put_factor<2>(R, m, r0, c0, beta);
    }
    __syncthreads();
    if (warp >= 2) {    // 32 -> 64: this warp's rows, columns 0-31
        const int r0 = 16 * warp;
        float m[4][4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                m[x][v] = acc[x][v];
        minus_product<32, 4>(m, L, R, r0, 0, 0);
        put_factor<4>(R, m, r0, 0, beta);
        asm volatile("bar.sync 1, 64;" ::: "memory");
        minus_product<32, 4>(m, L, R, r0, 32, 0);
        put_factor<4>(L, m, r0, 0, nullptr);
    }
    __syncthreads();
    // hi and lo as 128B-swizzled rows, the shared-memory image that the sweeps load
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        const int lo = x >> 2, i = (tid >> 3) + 16 * (x & 3), c16 = tid & 7;
        *reinterpret_cast<uint4 *>(sc.b + tile * BTILE + lo * (BTILE / 2) + i * 128 +
                                   ((c16 ^ (i & 7)) << 4)) =
            *reinterpret_cast<const uint4 *>(&L[lo][i][8 * c16]);
    }
}

// ---- the sweeps -----------------------------------------------------------------
//
// 608 threads: warp 0 loads, warp 1 issues the products, warps 2-9 ("chain") carry X,
// the state's operand and the state between products, each a quarter of the lanes and
// half of the columns, warps 10-17 ("side") do what the chain does not wait for (P,
// beta Eps, O; back: P, scale e^G Q, dO^T) and warp 18 sends out what they leave in
// shared memory: as stores of these warps it would stand before the chain's own
// accesses to shared memory and TMEM.
// Q and K of a chunk lie as one 128-row tile: [Q; K] K^T gives the scores in lanes
// 0-63 (lanes 64-127, K K^T, are not used).

constexpr int SWEEP = 608;
constexpr int CHAIN = 256, SIDE = 256;
constexpr int NS = 2, NT = 4;                   // stages; of the tables
constexpr int QK = 0, VD = 32768, BB = 49152, STAGE = 65536;
constexpr int POFF = NS * STAGE;                // P hi, lo: [64][64] bf16 each
constexpr int QOFF = POFF + 16384;              // backward: scale e^G Q, hi, lo
constexpr int Q2 = 16384;                       // bytes of one of them: [2][64][64] bf16
template <bool BWD> struct SweepLayout {
    static constexpr int SOFF = QOFF + (BWD ? 2 * Q2 : 0);     // the state's image on its way out
    static constexpr int OOFF = SOFF + STILE;                       // O on its way out
    static constexpr int TOFF = OOFF + (BWD ? 0 : 16384);
    static constexpr int MOFF = TOFF + NT * TAB;
    static constexpr int NBAR = 4 * NS + 2 * NT + 18 + 2 * NS + 2;
    static constexpr int SLOT = MOFF + NBAR * 8;
    static constexpr int ABORT = SLOT + 4;
    static constexpr int RANK = ABORT + 4;
    static constexpr int DYN = RANK + 4 + 1024;
    static_assert(DYN <= 232448, "shared memory per CTA");
};
// TMEM columns: the state fp32, its hi and lo; forward: O's inter term, the chain's
// accumulator, scores and then O's intra term; back: scores and then P^T dO, the
// chain's accumulator, dO^T of two chunks; the chain's operand (beta X, then kappa
// beta Eps), hi and lo
constexpr uint32_t TS = 0, TSH = 128, T2 = 256, T1 = 320, TR = 384, TD = 384, TY = 448,
                   TCOLS = 512;
// an operand of 64 tokens in 64 columns: for each half of the tokens 16 columns of
// hi, 16 of lo, so that the threads of a half write among columns of their own
__device__ __forceinline__ uint32_t tok_col(int kk, int lo)
{
    return 32 * (kk >> 1) + 8 * (kk & 1) + 16 * lo;
}

struct SweepParams {
    CUtensorMap mq, mk, mv, mo;     // mv: v, or back: do; mo: o, where a.o is given, or back: dv
    DeltaArgs a;
    Scratch sc;
    int segs, seg_len;  // segments of a sequence (1: whole), their tokens: whole chunks
    int states;         // the states alone, of a segment from zero, and (forward) Phi
};

// 32 values a lane (this lane's channel, 32 tokens) to bf16 rows, a token a row:
// neighbouring lanes trade, each stores a pair of channels of every other token, the
// even lane from the first on.  at: the lane's first row (its pair), step: bytes from
// there to the row after next; n: rows there are, from this half's first on.
__device__ __forceinline__ void store_rows(const float (&x)[32], bool odd, uint8_t *at,
                                           int64_t step, int n)
{
#pragma unroll
    for (int m = 0; m < 16; ++m) {
        const float mine = odd ? x[2 * m + 1] : x[2 * m], other = odd ? x[2 * m] : x[2 * m + 1];
        const float got = __shfl_xor_sync(0xffffffffu, other, 1);
        const uint32_t pair = odd ? pack_bf16x2(got, mine) : pack_bf16x2(mine, got);
        if (2 * m + odd < n)
            *reinterpret_cast<uint32_t *>(at) = pair;
        at += step;
    }
}
// to a [2][64 tokens][64 channels] swizzled tile
__device__ __forceinline__ void store_image(const float (&x)[32], int half, int e, uint8_t *tile)
{
    const bool odd = e & 1;
    uint8_t *at = tile + (e >> 6) * 8192 + (32 * half + odd) * 128 + (e & 6) * 2;
    const int c16 = (e & 63) >> 3;
#pragma unroll
    for (int m = 0; m < 16; ++m) {
        const float mine = odd ? x[2 * m + 1] : x[2 * m], other = odd ? x[2 * m] : x[2 * m + 1];
        const float got = __shfl_xor_sync(0xffffffffu, other, 1);
        const uint32_t pair = odd ? pack_bf16x2(got, mine) : pack_bf16x2(mine, got);
        *reinterpret_cast<uint32_t *>(at + m * 256 + ((c16 ^ ((2 * m + odd) & 7)) << 4)) = pair;
    }
}
// Channel e of tokens 32 half .. of a [2][64 tokens][64 channels] swizzled tile,
// pairs of tokens packed.
__device__ __forceinline__ void channel(const uint8_t *tile, int e, int half, uint32_t (&v)[16])
{
    const uint8_t *at = tile + (e >> 6) * 8192 + 32 * half * 128 + (e & 7) * 2;
    const int c16 = (e & 63) >> 3;
#pragma unroll
    for (int x = 0; x < 32; ++x) {
        const uint32_t b =
            *reinterpret_cast<const uint16_t *>(at + x * 128 + ((c16 ^ (x & 7)) << 4));
        v[x / 2] = x & 1 ? v[x / 2] | b << 16 : b;
    }
}
template <bool BWD>
__global__ void __launch_bounds__(SWEEP, 1)
    delta_sweep_kernel(const __grid_constant__ SweepParams P)
{
    using L = SweepLayout<BWD>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *sm = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~static_cast<uintptr_t>(1023));
    const DeltaArgs &a = P.a;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + L::MOFF);    // Q, K
    uint64_t *fullv = full + NS, *fullb = full + 2 * NS, *empty = full + 3 * NS;
    uint64_t *tfull = full + 4 * NS, *tempty = tfull + NT;          // tables
    uint64_t *bars = tempty + NT;
    uint64_t *sc_full = bars;           // scores (and Q S)
    uint64_t *ks_full = bars + 1;       // K S (back: K K', and P^T dO)
    uint64_t *e_full = bars + 2;        // Eps (R)
    uint64_t *s_full = bars + 3;        // the state
    uint64_t *o_full = bars + 4;        // O
    uint64_t *s_ready = bars + 5;       // the state's hi, lo and its decayed fp32
    uint64_t *y_ready = bars + 6;       // X and beta X
    uint64_t *w_ready = bars + 7;       // what the state takes
    uint64_t *p_ready = bars + 8;       // P
    uint64_t *q_ready = bars + 9;       // Q S read out of TMEM; back: scale e^G Q
    uint64_t *r_ready = bars + 10;      // O's intra term read
    uint64_t *d_ready = bars + 11;      // beta Eps
    uint64_t *i_ready = bars + 12;      // the state's image
    uint64_t *i_free = bars + 13;       // it has been read
    uint64_t *o_ready = bars + 14;      // O in shared memory
    uint64_t *o_free = bars + 15;       // it has been read
    uint64_t *x_read = bars + 16;       // forward: Eps read by the side warps
    uint64_t *drain = bars + 17;
    // These take turns by chunk: what arrives for the next chunk does not wait until its
    // waiter has seen this one, and a waiter that comes a phase late waits for good.
    uint64_t *e_ready = bars + 18;              // [NS] Eps's (R's) image
    uint64_t *e_free = bars + 18 + NS;          // [NS] it has been read
    uint64_t *td_ready = bars + 18 + 2 * NS;    // [2] back: dO^T in TMEM
    uint32_t *tslot = reinterpret_cast<uint32_t *>(sm + L::SLOT);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(sm + L::ABORT);
    volatile int *rank_slot = reinterpret_cast<volatile int *>(sm + L::RANK);
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&fullv[i], 1);
            mbar_init(&fullb[i], 1);
            mbar_init(&empty[i], 1);
            mbar_init(&e_ready[i], SIDE / 32);
            mbar_init(&e_free[i], 1);
        }
        for (int i = 0; i < NT; ++i) {
            mbar_init(&tfull[i], 1);
            // the forward's side warps have nothing to do for the states alone
            mbar_init(&tempty[i], CHAIN / 32 + (!BWD && P.states ? 0 : SIDE / 32));
        }
        for (int i = 0; i < 5; ++i)
            mbar_init(&bars[i], 1);
        mbar_init(s_ready, CHAIN / 32);
        mbar_init(y_ready, CHAIN / 32);
        mbar_init(w_ready, CHAIN / 32);
        mbar_init(p_ready, SIDE / 64);
        mbar_init(q_ready, BWD ? SIDE / 64 : SIDE / 32);
        mbar_init(d_ready, CHAIN / 32);
        mbar_init(x_read, SIDE / 32);
        mbar_init(i_ready, CHAIN / 32);
        mbar_init(o_ready, SIDE / 32);
        mbar_init(o_free, 1);
        mbar_init(i_free, 1);
        mbar_init(&td_ready[0], SIDE / 32);
        mbar_init(&td_ready[1], SIDE / 32);
        mbar_init(r_ready, SIDE / 32);
        mbar_init(drain, 1);
        *abort_flag = 0;
        *rank_slot = blockIdx.x / a.H;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tslot, TCOLS);
        tmem_relinquish();
    }
    if (warp == 0 && lane == 0) {
        prefetch_tmap(&P.mq);
        prefetch_tmap(&P.mk);
        prefetch_tmap(&P.mv);
        if (BWD || a.o.p)
            prefetch_tmap(&P.mo);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tslot;
    const int h = blockIdx.x % a.H;
    const bool states = P.states;
    // Phi's sweep: no values, from the identity, D columns
    const bool phi = !BWD && states && blockIdx.y == 1;
    // packed sequences the longest first: a late long one would run alone.  Each
    // CTA counts for itself which it is (N * N compares over 608 threads).
    if (a.cu && a.N > 1 && a.N <= 256 && P.segs == 1) {
        const int rank = blockIdx.x / a.H;
        for (int n = threadIdx.x; n < a.N; n += SWEEP) {
            const int len = a.cu[n + 1] - a.cu[n];
            int before = 0;
            for (int m = 0; m < a.N; ++m) {
                const int other = a.cu[m + 1] - a.cu[m];
                before += other > len || (other == len && m < n);
            }
            if (before == rank)
                *rank_slot = n;
        }
        __syncthreads();
    }
    const int seg = *rank_slot % P.segs;
    Seq sq = sequence(a.cu, a.T, *rank_slot / P.segs);
    // whether the sequence's state leaves this segment (back: its first one)
    bool last = true;
    if (P.segs > 1) {
        const int64_t from = (int64_t)seg * P.seg_len;
        last = BWD ? seg == 0 : from + P.seg_len >= sq.len;
        // nothing to do: past the end (segment 0 carries an empty sequence's state on),
        // or a state that no segment takes (the last Phi is the backward's)
        if ((seg > 0 && from >= sq.len) || (states && last && !(phi && P.sc.s)))
            sq.len = -1;
        else
            sq.len = min(sq.len - from, (int64_t)P.seg_len);
        sq.bos += from;
        sq.slot += from / C;
    }
    const bool idle = sq.len < 0;
    const int nc = idle ? 0 : (int)((sq.len + C - 1) / C);
    // c counts chunks in the order of the sweep
    auto chunk = [&](int c) { return BWD ? nc - 1 - c : c; };
    auto tokens = [&](int c) { return (int)min((int64_t)C, sq.len - (int64_t)chunk(c) * C); };
    auto tile_of = [&](int c) { return (sq.slot + chunk(c)) * a.H + h; };
    const float *tabs = reinterpret_cast<const float *>(sm + L::TOFF);
    const bool keep = !states && (BWD || P.sc.s);   // the images are wanted
    // O (dV) leaves tile by tile; the last rows of a packed sequence row by row, the rows
    // after them are another's
    const bool some_o = !BWD && a.o.p && !states;
    auto o_tile = [&](int c) { return !a.cu || tokens(c) == C; };
    // this lane's first row of 32 from token j0 of the chunk, at its pair of channels
    auto token_rows = [&](const TokOut &o, int c, int j0, int e) {
        return reinterpret_cast<uint8_t *>(
            static_cast<__nv_bfloat16 *>(o.p) + sq.row * o.sb +
            (sq.bos + (int64_t)chunk(c) * C + j0 + (lane & 1)) * o.st + (int64_t)h * o.sh +
            (e & ~1));
    };

    if (warp == 0) {
        // ------------------------------------------------------------- loads
        if (lane == 0) {
            const int hq = h / a.q.hdiv;
            int issued = 0, tables = 0;
            bool going = true;
            auto tables_in = [&]() {
                const int ts = tables % NT;
                if (tables >= NT &&
                    !(going = wait_call(&tempty[ts], (tables / NT - 1) & 1, abort_flag)))
                    return false;
                mbar_arrive_expect_tx(&tfull[ts], TAB);
                bulk_load(sm + L::TOFF + ts * TAB, P.sc.tab + tile_of(tables) * TABS * C, TAB,
                          &tfull[ts]);
                ++tables;
                return true;
            };
#pragma unroll 1
            for (int c = 0; c < nc; ++c) {
                const int s = c % NS;
                // tables a chunk ahead, the tiles of the chunk after this into L2: its
                // stage is free a chunk later
                while (tables < nc && tables < c + 2 && tables_in())
                    ;
                if (!going)
                    break;
                if (c >= NS) {
                    // Eps's (R's) image lies where V (dO) was, dV's where Q was
                    if (!(going = (!keep || wait_call(&e_free[s], (c / NS - 1) & 1, abort_flag)) &&
                                  wait_call(&empty[s], (c / NS - 1) & 1, abort_flag)))
                        break;
                }
                const int t = (int)(sq.bos + (int64_t)chunk(c) * C);
                uint8_t *st = sm + s * STAGE;
                mbar_arrive_expect_tx(&full[s], 32768);
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    tma_load_4d(st + QK + b * 16384, &P.mq, &full[s], 64 * b, hq, t, (int)sq.row);
                    tma_load_4d(st + QK + b * 16384 + 8192, &P.mk, &full[s], 64 * b, hq, t,
                                (int)sq.row);
                }
                mbar_arrive_expect_tx(&fullv[s], 16384);
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    tma_load_4d(st + VD + b * 8192, &P.mv, &fullv[s], 64 * b, h, t, (int)sq.row);
                mbar_arrive_expect_tx(&fullb[s], BTILE);
                bulk_load(st + BB, P.sc.b + tile_of(c) * BTILE, BTILE, &fullb[s]);
                if (const int c1 = c + (c == 0 ? 1 : 2); c1 < nc) {
                    const int t1 = (int)(sq.bos + (int64_t)chunk(c1) * C);
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
                        tma_prefetch_l2_4d(&P.mq, 64 * b, hq, t1, (int)sq.row);
                        tma_prefetch_l2_4d(&P.mk, 64 * b, hq, t1, (int)sq.row);
                        tma_prefetch_l2_4d(&P.mv, 64 * b, h, t1, (int)sq.row);
                    }
                    bulk_prefetch(P.sc.b + tile_of(c1) * BTILE, BTILE);
                }
                ++issued;
            }
            for (int c = issued > NS ? issued - NS : 0; c < issued; ++c) {
                drain_wait(&full[c % NS], (c / NS) & 1);
                drain_wait(&fullv[c % NS], (c / NS) & 1);
                drain_wait(&fullb[c % NS], (c / NS) & 1);
            }
            for (int c = tables > NT ? tables - NT : 0; c < tables; ++c)
                drain_wait(&tfull[c % NT], (c / NT) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------- products
        const uint32_t sb = smem_u32(sm);
        constexpr uint32_t id64 = idesc_bf16_f32(128, 64, 0, 0);       // B K-major
        constexpr uint32_t id64mn = idesc_bf16_f32(128, 64, 0, 1);     // B MN-major
        constexpr uint32_t id128mn = idesc_bf16_f32(128, 128, 0, 1);
        // Descriptors of stage 0 once; another place is an addition to the address
        // field (16-byte units): what one product costs to issue counts here.
        const uint64_t d_rows = sdesc_sw128(sb + QK, 16, 1024);        // [Q; K] by rows
        const uint64_t d_cols = sdesc_sw128(sb + QK, 16384, 1024);     // D along M or N
        const uint64_t d_b = sdesc_sw128(sb + BB, 16, 1024);
        const uint64_t d_bmn = sdesc_sw128(sb + BB, 8192, 1024);
        const uint64_t d_p = sdesc_sw128(sb + POFF, 16, 1024);
        const uint64_t d_pmn = sdesc_sw128(sb + POFF, 8192, 1024);
        const uint64_t d_q2 = sdesc_sw128(sb + QOFF, 8192, 1024);
        auto off = [](uint32_t bytes) { return (uint64_t)(bytes >> 4); };
        auto stage = [&](int c) { return off((uint32_t)((c % NS) * STAGE)); };
        // k-step kk of D in a tile of 128 rows
        auto kd = [&](int kk) { return off((uint32_t)((kk >> 2) * 16384 + (kk & 3) * 32)); };
        auto scores = [&](int c) {      // [Q; K] K^T
            const uint64_t d = d_rows + stage(c);
#pragma unroll 1
            for (int k4 = 0; k4 < 2; ++k4)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ss(tm + (BWD ? T2 : TR), d + kd(4 * k4 + kk),
                           d + off(8192) + kd(4 * k4 + kk), id64, k4 + kk > 0);
            mma_commit(sc_full);
        };
        // the state's rows times those of the [Q; K] tile from `row` on
        auto state_times = [&](uint32_t to, int c, int row) {
            const uint64_t d = d_rows + stage(c) + off(row * 128);
#pragma unroll 1
            for (int k4 = 0; k4 < 4; ++k4)      // hi's D, then lo's
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ts(tm + to, tm + TSH + 32 * k4 + 8 * kk, d + kd((4 * k4 + kk) & 7), id64,
                           k4 + kk > 0);
        };
        // T1 += (beta X)^T B^T (back: B): hi hi, lo hi, hi lo
        auto solve = [&](int c) {
            const uint64_t d = (BWD ? d_bmn : d_b) + stage(c);
#pragma unroll 1
            for (int x = 0; x < 3; ++x)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ts(tm + T1, tm + TY + tok_col(kk, x == 1),
                           d + off((x == 2 ? BTILE / 2 : 0) + kk * (BWD ? 2048 : 32)),
                           BWD ? id64mn : id64, 1);
            mma_commit(e_full);
        };
        // the state += (chain's operand)^T K
        auto update = [&](int c) {
            const uint64_t d = d_cols + stage(c) + off(8192);
#pragma unroll 1
            for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    mma_ts(tm + TS, tm + TY + tok_col(kk, lo), d + off(kk * 2048), id128mn, 1);
            mma_commit(s_full);
        };
        // The tokens past a packed sequence's end are another's: zeros in their
        // place (the loads fill with zeros past the tensor's end).
        auto clear_tail = [&](int c) {
            if (!a.cu || chunk(c) != nc - 1)
                return true;
            const int n = tokens(c);
            if (!warp_all(wait_call(&fullv[c % NS], (c / NS) & 1, abort_flag)))
                return false;
            uint8_t *st = sm + (c % NS) * STAGE;
            const uint4 z = make_uint4(0, 0, 0, 0);
            for (int x = lane; x < (C - n) * 8; x += 32) {
                const int off = (n + x / 8) * 128 + (x % 8) * 16;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    *reinterpret_cast<uint4 *>(st + QK + b * 8192 + off) = z;
#pragma unroll
                for (int b = 0; b < 2; ++b)
                    *reinterpret_cast<uint4 *>(st + VD + b * 8192 + off) = z;
            }
            fence_proxy_async_smem();
            __syncwarp();
            return true;
        };
        auto stage_in = [&](int c) {
            return warp_all(wait_call(&full[c % NS], (c / NS) & 1, abort_flag) &&
                            wait_call(&fullb[c % NS], (c / NS) & 1, abort_flag)) &&
                   clear_tail(c);
        };
        auto both = [&](uint64_t *bar, int c) {
            const bool ok = warp_all(wait_call(bar, c & 1, abort_flag));
            tc_fence_after();
            return ok;
        };
        const bool one = elect_one();
        bool any = false;
        if (BWD && nc > 0 && stage_in(0)) {
            any = true;
            if (one)
                scores(0);
            __syncwarp();
            // dO^T goes in from TMEM: as an A operand in shared memory it would lie
            // MN-major (delta_grads was slower with such operands)
            auto prior = [&](int c) {   // dO^T P
                if (!both(p_ready, c) || !both(&td_ready[c & 1], c >> 1))
                    return false;
                if (one)
#pragma unroll 1
                    for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ts(tm + T2, tm + TD + 32 * (c & 1) + 8 * kk,
                                   d_pmn + off(lo * 8192 + kk * 2048), id64mn, lo + kk > 0);
                __syncwarp();
                return true;
            };
            bool ok = prior(0);
#pragma unroll 1
            for (int c = 0; ok && c < nc; ++c) {
                if (!(ok = both(s_ready, c)))
                    break;
                if (one) {
                    state_times(T1, c, 64);
                    mma_commit(ks_full);
                }
                __syncwarp();
                // what the chain does not wait for goes between its products, while its
                // warps work
                if (!(ok = both(q_ready, c)))
                    break;
                if (one)    // K'^T += dO^T (scale e^G Q)
#pragma unroll 1
                    for (int lo = 0; lo < 2; ++lo)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ts(tm + TS, tm + TD + 32 * (c & 1) + 8 * kk,
                                   d_q2 + off(lo * Q2 + kk * 2048), id128mn, 1);
                __syncwarp();
                if (!(ok = both(y_ready, c)))
                    break;
                if (one)
                    solve(c);
                __syncwarp();
                if (c + 1 < nc) {   // over dO^T P, which W has taken
                    if (!(ok = stage_in(c + 1)))
                        break;
                    if (one)
                        scores(c + 1);
                    __syncwarp();
                }
                if (!(ok = both(w_ready, c)))
                    break;
                if (one) {
                    update(c);
                    mma_commit(&empty[c % NS]);
                }
                __syncwarp();
                if (c + 1 < nc)
                    ok = prior(c + 1);
            }
        } else if (!BWD && nc > 0 && stage_in(0)) {
            any = true;
#pragma unroll 1
            for (int c = 0; c < nc; ++c) {
                if (!both(s_ready, c))
                    break;
                if (one) {
                    state_times(T1, c, 64);
                    mma_commit(ks_full);
                }
                __syncwarp();
                // what the chain does not wait for goes between its products, while its
                // warps work: Q S and the scores while X is made, O's intra term while
                // S is
                if (!states) {
                    if (c > 0 && (!both(q_ready, c - 1) || !both(r_ready, c - 1)))
                        break;
                    if (one) {
                        state_times(T2, c, 0);
                        scores(c);
                    }
                    __syncwarp();
                }
                if (!both(y_ready, c))
                    break;
                if (one)
                    solve(c);
                __syncwarp();
                if ((c + 1 < nc && !stage_in(c + 1)) || !both(w_ready, c))
                    break;
                if (one) {
                    update(c);
                    mma_commit(&empty[c % NS]);
                }
                __syncwarp();
                if (states)
                    continue;
                if (!both(p_ready, c) || !both(d_ready, c))
                    break;
                if (one) {  // (beta Eps)^T P^T; beta Eps lies in T1, as tok_col
#pragma unroll 1
                    for (int x = 0; x < 3; ++x)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ts(tm + TR, tm + T1 + tok_col(kk, x == 1),
                                   d_p + off((x == 2 ? 8192 : 0) + kk * 32), id64, x + kk > 0);
                    mma_commit(o_full);
                }
                __syncwarp();
            }
        }
        if (any && one) {   // every product is done before TMEM is released
            mma_commit(drain);
            drain_wait(drain, 0);
            if (!mbar_try_wait(drain, 0))   // it never came: waits without a clock end too
                *abort_flag = 1;
        }
        __syncwarp();
    } else if (warp == 18) {
        // ------------------------------------------------------------ stores
        if (lane == 0) {
            uint8_t *simg = BWD ? P.sc.k : P.sc.s, *eimg = BWD ? P.sc.r : P.sc.e;
#pragma unroll 1
            for (int c = 0; c < nc; ++c) {
                if (keep) {
                    if (!wait_call(i_ready, c & 1, abort_flag))
                        break;
                    bulk_store(simg + tile_of(c) * STILE, sm + L::SOFF, STILE);
                    bulk_commit_group();
                    bulk_wait_read_all();
                    mbar_arrive(i_free);
                    if (!wait_call(&e_ready[c % NS], (c / NS) & 1, abort_flag))
                        break;
                    const uint8_t *st = sm + (c % NS) * STAGE;
                    bulk_store(eimg + tile_of(c) * ETILE, st + VD, ETILE);
                    if (BWD && o_tile(c)) {
                        const int t = (int)(sq.bos + (int64_t)chunk(c) * C);
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            if (64 * b < a.E)
                                tma_store_4d(&P.mo, st + QK + b * 16384, 64 * b, h, t, (int)sq.row);
                    }
                    bulk_commit_group();
                    bulk_wait_read_all();
                    mbar_arrive(&e_free[c % NS]);
                }
                if (some_o) {
                    if (!wait_call(o_ready, c & 1, abort_flag))
                        break;
                    if (o_tile(c)) {
                        const int t = (int)(sq.bos + (int64_t)c * C);
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            if (64 * b < a.E)
                                tma_store_4d(&P.mo, sm + L::OOFF + b * 8192, 64 * b, h, t,
                                             (int)sq.row);
                        bulk_commit_group();
                        bulk_wait_read_all();
                    }
                    mbar_arrive(o_free);
                }
            }
        }
        __syncwarp();
    } else if (warp < 10) {
        // ------------------------------------------------------------- chain
        const int q = warp & 3, half = (warp - 2) >> 2;
        const int e = 32 * q + lane;
        const uint32_t lanes = tm + ((uint32_t)(32 * q) << 16);
        // states [.][H][D][E], of sequences or of segments (Phi: [.][H][D][D])
        const int E = phi ? a.D : a.E;
        const int64_t one_state = (int64_t)a.D * E;
        const int64_t at_seq = ((int64_t)sq.n * a.H + h) * one_state;
        const int64_t at_seg = ((int64_t)blockIdx.x / a.H * a.H + h) * one_state;
        const float *in = BWD ? a.dfin : a.init;
        float *out = BWD ? a.dinit : a.fin;
        if (in)
            in += at_seq;
        if (out)
            out += at_seq;
        if (states) {
            in = nullptr;
            out = (phi ? P.sc.phi : P.sc.own) + at_seg;
        } else if (P.segs > 1) {
            in = P.sc.enter + at_seg;
            out = last ? out : nullptr;
        }
        if (idle)
            out = nullptr;
        bool ok = true;
        if (nc > 0)
#pragma unroll 1
            for (int d0 = 64 * half; d0 < 64 * half + 64; d0 += 32) {
                uint32_t r[32];     // the loads all at once
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    r[x] = in && e < E && d0 + x < a.D
                               ? __float_as_uint(in[(int64_t)(d0 + x) * E + e])
                               : phi && e == d0 + x && e < a.D ? __float_as_uint(1.f) : 0u;
                tmem_st32_issue(lanes + TS + d0, r);
                tmem_wait_st();
            }
#pragma unroll 1
        for (int c = 0; ok && c < nc; ++c) {
            const int s = c % NS, n = tokens(c);
            const uint8_t *st = sm + s * STAGE;
            const float *tab = tabs + (c % NT) * TABS * C;
            if (!(ok = warp_all(wait_role<BWD>(&tfull[c % NT], (c / NT) & 1, abort_flag))))
                break;
            // ---- the state
            if (c > 0 && !(ok = warp_all(wait_role<BWD>(s_full, (c - 1) & 1, abort_flag))))
                break;
            tc_fence_after();
            const float2 gC = make_float2(-tab[TNEG * C + C - 1], -tab[TNEG * C + C - 1]);
#pragma unroll 1
            for (int d0 = 64 * half; d0 < 64 * half + 64; d0 += 32) {
                uint32_t r[32], hi[16], lo[16];
                tmem_ld32(lanes + TS + d0, r);
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    split2(pair_of(r, x), hi[x], lo[x]);
                    put_pair(r, x, mul2(gC, pair_of(r, x)));
                }
                tmem_st16_issue(lanes + TSH + d0 / 2, hi);
                tmem_st16_issue(lanes + TSH + 64 + d0 / 2, lo);
                tmem_st32_issue(lanes + TS + d0, r);
            }
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(s_ready);
            if (keep) {
                if (c > 0 && !(ok = warp_all(wait_role<BWD>(i_free, (c - 1) & 1, abort_flag))))
                    break;
                // hi, back from TMEM
                uint8_t *to = sm + L::SOFF + half * 16384 + e * 128;
#pragma unroll 1
                for (int p = 0; p < 2; ++p) {
                    uint32_t hi[16];
                    tmem_ld16(lanes + TSH + 32 * half + 16 * p, hi);
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        *reinterpret_cast<uint4 *>(to + (((4 * p + x) ^ (e & 7)) << 4)) =
                            make_uint4(hi[4 * x], hi[4 * x + 1], hi[4 * x + 2], hi[4 * x + 3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(i_ready);
            }
            // ---- X (W)
            const int j0 = 32 * half;
            const float *tj = tab + j0;
            auto pair_at = [&](int which, int m) {
                return *reinterpret_cast<const float2 *>(tj + which * C + 2 * m);
            };
            uint32_t v[16];
            if constexpr (!BWD) {
                if (!(ok = warp_all(wait_role<BWD>(&fullv[s], (c / NS) & 1, abort_flag))))
                    break;
                channel(st + VD, e, half, v);
                if (phi)
#pragma unroll
                    for (int x = 0; x < 16; ++x)
                        v[x] = 0u;
            }
            if (!(ok = warp_all(wait_role<BWD>(ks_full, c & 1, abort_flag))))
                break;
            tc_fence_after();
            uint32_t r[32], hi[16], lo[16];
            if constexpr (BWD) {
                uint32_t p[32];
                tmem_ld32_issue(lanes + T1 + j0, r);
                tmem_ld32_issue(lanes + T2 + j0, p);
                tmem_wait_ld(r, p);
#pragma unroll
                for (int x = 0; x < 16; ++x)
                    put_pair(r, x, fma2(pair_at(TKAP, x), pair_of(r, x), pair_of(p, x)));
            } else {
                tmem_ld32(lanes + T1 + j0, r);
#pragma unroll
                for (int x = 0; x < 16; ++x)
                    put_pair(r, x, fma2(pair_at(TNEG, x), pair_of(r, x),
                                        make_float2(bf16lo(v[x]), bf16hi(v[x]))));
            }
            if (n < C)
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    if (j0 + x >= n)
                        r[x] = 0u;
#pragma unroll
            for (int x = 0; x < 16; ++x)
                split2(mul2(pair_at(TNB, x), pair_of(r, x)), hi[x], lo[x]);
            tmem_st32_issue(lanes + T1 + j0, r);
            tmem_st16_issue(lanes + TY + 32 * half, hi);
            tmem_st16_issue(lanes + TY + 32 * half + 16, lo);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0 && !(a.withhold_handoff && c == 0 && warp == 2))
                mbar_arrive(y_ready);
            // ---- Eps (R)
            if (!(ok = warp_all(wait_role<BWD>(e_full, c & 1, abort_flag))))
                break;
            tc_fence_after();
            tmem_ld32(lanes + T1 + j0, r);
#pragma unroll
            for (int x = 0; x < 16; ++x)
                split2(mul2(pair_at(BWD ? TNGB : TKB, x), pair_of(r, x)), hi[x], lo[x]);
            tmem_st16_issue(lanes + TY + 32 * half, hi);
            tmem_st16_issue(lanes + TY + 32 * half + 16, lo);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(w_ready);
            // off the chain, while the state is made.  Back: R's image, and dV from R before
            // its rounding, where Q was: the scores and scale e^G Q are done with it
            if (BWD && keep) {
                float x32[32];
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    x32[x] = __uint_as_float(r[x]);
                store_image(x32, half, e, sm + s * STAGE + VD);
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const float2 y = mul2(pair_at(TBETA, x), pair_of(r, x));
                    x32[2 * x] = y.x;
                    x32[2 * x + 1] = y.y;
                }
                if (o_tile(c))
                    store_image(x32, half, e, sm + s * STAGE + QK + (e >> 6) * 8192);
                else
                    store_rows(x32, lane & 1, token_rows(a.dv, c, j0, e), 4 * a.dv.st,
                               e < a.E ? n - j0 : 0);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&e_ready[s]);
            }
            // forward: beta Eps over this half's own columns of T1, for O
            if (!BWD && !states) {
                // r is Eps still
#pragma unroll
                for (int x = 0; x < 16; ++x)
                    split2(mul2(pair_at(TBETA, x), pair_of(r, x)), hi[x], lo[x]);
                // the side warps have read Eps, where they want it
                if (keep && !(ok = warp_all(wait_role<BWD>(x_read, c & 1, abort_flag))))
                    break;
                tmem_st16_issue(lanes + T1 + 32 * half, hi);
                tmem_st16_issue(lanes + T1 + 32 * half + 16, lo);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(d_ready);
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&tempty[c % NT]);
        }
        if (ok && nc > 0)
            ok = warp_all(wait_role<BWD>(s_full, (nc - 1) & 1, abort_flag));
        tc_fence_after();
        if (ok && out)
#pragma unroll 1
            for (int d0 = 64 * half; d0 < 64 * half + 64; d0 += 8) {
                uint32_t r[8];
                if (nc > 0)
                    tmem_ld8(lanes + TS + d0, r);
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    if (e < E && d0 + x < a.D) {
                        const int64_t at = (int64_t)(d0 + x) * E + e;
                        out[at] = nc > 0 ? __uint_as_float(r[x]) : in ? in[at] : 0.f;
                    }
            }
    } else {
        // -------------------------------------------------------------- side
        const int q = warp & 3, half = (warp - 10) >> 2;
        const int row = 32 * q + lane;
        const uint32_t lanes = tm + ((uint32_t)(32 * q) << 16);
        const int j0 = 32 * half;
        const int todo = !BWD && states ? 0 : nc;
#pragma unroll 1
        for (int c = 0; c < todo; ++c) {
            const int s = c % NS, n = tokens(c);
            const float *tab = tabs + (c % NT) * TABS * C;
            if constexpr (BWD) {    // dO^T: this lane's channel, this half's tokens
                if (!warp_all(wait_role<BWD>(&fullv[s], (c / NS) & 1, abort_flag)))
                    break;
                uint32_t v[16];
                channel(sm + s * STAGE + VD, row, half, v);
                if (n < C)
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        if (j0 + 2 * x >= n)
                            v[x] = 0u;
                        else if (j0 + 2 * x + 1 >= n)
                            v[x] &= 0xFFFFu;
                    }
                tmem_st16_issue(lanes + TD + 32 * (c & 1) + 16 * half, v);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&td_ready[c & 1]);
            }
            if (!warp_all(wait_role<BWD>(&tfull[c % NT], (c / NT) & 1, abort_flag)) ||
                !warp_all(wait_role<BWD>(sc_full, c & 1, abort_flag)))
                break;
            tc_fence_after();
            if (q < 2) {    // row i of P, this half's columns; those past the warp's rows are zero
                const int i = row;
                uint8_t *to = sm + POFF + i * 128;
                uint32_t hi[16] = {}, lo[16] = {};
                if (half <= q) {
                    const float gi = tab[TLOG * C + i], li = tab[TLOW * C + i];
                    const float2 gi2 = make_float2(gi, gi), li2 = make_float2(li, li);
                    const float2 s2 = make_float2(a.scale, a.scale);
                    const float2 minus = make_float2(-1.f, -1.f);
                    uint32_t r[32];
                    tmem_ld32(lanes + (BWD ? T2 : TR) + j0, r);
                    const float *gj = tab + TLOG * C + j0, *lj = tab + TLOW * C + j0;
#pragma unroll
                    for (int x = 0; x < 16; ++x) {
                        const float2 d = add2(
                            fma2(*reinterpret_cast<const float2 *>(gj + 2 * x), minus, gi2),
                            fma2(*reinterpret_cast<const float2 *>(lj + 2 * x), minus, li2));
                        float2 y = mul2(mul2(make_float2(exp2_fast(d.x), exp2_fast(d.y)), s2),
                                        pair_of(r, x));
                        if (half == q) {
                            y.x = 2 * x <= lane ? y.x : 0.f;
                            y.y = 2 * x + 1 <= lane ? y.y : 0.f;
                        }
                        split2(y, hi[x], lo[x]);
                    }
                }
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint8_t *at = to + (((4 * half + x) ^ (i & 7)) << 4);
                    *reinterpret_cast<uint4 *>(at) =
                        make_uint4(hi[4 * x], hi[4 * x + 1], hi[4 * x + 2], hi[4 * x + 3]);
                    *reinterpret_cast<uint4 *>(at + 8192) =
                        make_uint4(lo[4 * x], lo[4 * x + 1], lo[4 * x + 2], lo[4 * x + 3]);
                }
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(p_ready);
            } else if (BWD) {   // row i of scale e^G Q, this half's channels
                if (!warp_all(wait_role<BWD>(&full[s], (c / NS) & 1, abort_flag)))
                    break;
                const int i = row - 64;
                const float f = i < n ? -a.scale * tab[TNEG * C + i] : 0.f;
                const float2 f2 = make_float2(f, f);
                const uint8_t *from = sm + s * STAGE + QK + half * 16384 + i * 128;
                uint8_t *to = sm + QOFF + half * 8192 + i * 128;
#pragma unroll 4
                for (int x = 0; x < 8; ++x) {
                    const int off = (x ^ (i & 7)) << 4;
                    uint4 v = *reinterpret_cast<const uint4 *>(from + off);
                    if (i >= n)
                        v = make_uint4(0, 0, 0, 0);
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        split2(mul2(f2, make_float2(bf16lo(w[y]), bf16hi(w[y]))), hi[y], lo[y]);
                    *reinterpret_cast<uint4 *>(to + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(to + off + Q2) =
                        make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(q_ready);
            }
            // ---- the image of Eps, which delta_grads starts from
            if (!BWD && keep) {
                if (!warp_all(wait_role<BWD>(e_full, c & 1, abort_flag)))
                    break;
                tc_fence_after();
                uint32_t r[32];
                tmem_ld32(lanes + T1 + j0, r);
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(x_read);
                float x32[32];
#pragma unroll
                for (int x = 0; x < 32; ++x)
                    x32[x] = __uint_as_float(r[x]);
                store_image(x32, half, row, sm + s * STAGE + VD);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&e_ready[s]);
            }
            if constexpr (!BWD) {
                uint32_t inter[32], w[32];
                tmem_ld32(lanes + T2 + j0, inter);
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(q_ready);
                if (!warp_all(wait_role<BWD>(o_full, c & 1, abort_flag)))
                    break;
                tc_fence_after();
                tmem_ld32(lanes + TR + j0, w);
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(r_ready);
                const float2 s2 = make_float2(-a.scale, -a.scale);
                float y[32];
#pragma unroll
                for (int x = 0; x < 16; ++x) {
                    const float2 g =
                        *reinterpret_cast<const float2 *>(tab + TNEG * C + j0 + 2 * x);
                    const float2 z = fma2(mul2(g, s2), pair_of(inter, x), pair_of(w, x));
                    y[2 * x] = z.x;
                    y[2 * x + 1] = z.y;
                }
                if (some_o) {
                    if (c > 0 && !warp_all(wait_role<BWD>(o_free, (c - 1) & 1, abort_flag)))
                        break;
                    if (o_tile(c)) {
                        store_image(y, half, row, sm + L::OOFF);
                        fence_proxy_async_smem();
                    } else {
                        store_rows(y, lane & 1, token_rows(a.o, c, j0, row), 4 * a.o.st,
                                   row < a.E ? n - j0 : 0);
                    }
                    __syncwarp();
                    if (lane == 0)
                        mbar_arrive(o_ready);
                }
            }
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&tempty[c % NT]);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tm, TCOLS);
    }
}

// ---- dQ, dK, dg, dbeta --------------------------------------------------------------
//
// A CTA a (chunk, head), two of them an SM: 112 KB of tiles, 256 TMEM columns.  Lanes
// are tokens here: [dO; R] lie as one 128-row tile, as [Q; K] do, so that one product
// serves dQ (lanes 0-63) and dK's row part (lanes 64-127):
//     D1 = [scale e^G dO S^T; -e^G beta R S^T] + [W1; W2] K
//     DC = kappa beta Eps K'^T + [W1^T, W2^T] [Q; K]         (lanes 64-127)
// Every A operand is read along its rows (with MN-major ones 0.80 ms instead of 0.73
// at b4 h32 n8192, other things as they were then): W1 and W2 are written both ways, and DC's
// operands start 64 rows early, so that their rows meet lanes 64-127 where dK's other
// part is (lanes 0-63 of DC hold products of whatever lies before, read by nobody).

constexpr int GRADS = 256;
constexpr int GQ = 0, GE = 32768, GD = 49152, GS = 81920, GBAR = 114688;
constexpr int GW = GD, GWT = GD + 16384;        // over dO and R
constexpr int GTAB = GBAR + 64, GDYN = GTAB + 3 * C * 4;     // beta, G / ln 2
static_assert(TLOG == TBETA + 1 && TLOW == TLOG + 1 && 2 * (GDYN + 1024) <= 228 * 1024,
              "two CTAs an SM");
constexpr uint32_t U1 = 0, UC = 128, UW = 128, UCOLS = 256;

struct GradParams {
    CUtensorMap mq, mk, mdo;
    DeltaArgs a;
    Scratch sc;
};

// 32 numbers of a bf16 row (half a 128-byte row, 16-byte units c16 ..), as loaded
__device__ __forceinline__ float row_dot(const uint8_t *row, int i, int c0, const float (&x)[32])
{
    float t = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 v = *reinterpret_cast<const uint4 *>(row + (((c0 + c) ^ (i & 7)) << 4));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            t = fmaf(bf16lo(w[y]), x[8 * c + 2 * y], t);
            t = fmaf(bf16hi(w[y]), x[8 * c + 2 * y + 1], t);
        }
    }
    return t;
}
// 32 values to half of a swizzled 128-byte bf16 row
__device__ __forceinline__ void put_half_row(uint8_t *row, int i, int c0, const float (&x)[32])
{
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *reinterpret_cast<uint4 *>(row + (((c0 + c) ^ (i & 7)) << 4)) =
            make_uint4(pack_bf16x2(x[8 * c], x[8 * c + 1]), pack_bf16x2(x[8 * c + 2], x[8 * c + 3]),
                       pack_bf16x2(x[8 * c + 4], x[8 * c + 5]),
                       pack_bf16x2(x[8 * c + 6], x[8 * c + 7]));
}

__global__ void __launch_bounds__(GRADS, 2) delta_grads_kernel(const __grid_constant__ GradParams P)
{
    extern __shared__ __align__(1024) uint8_t sm[];
    const DeltaArgs &a = P.a;
    const int64_t slot = (int)blockIdx.x / a.H;
    const int h = (int)blockIdx.x - (int)slot * a.H;
    const Seq sq = sequence_of_slot(a.cu, a.T, a.N, slot);
    const int64_t t0 = (slot - sq.slot) * C;
    if (t0 >= sq.len)
        return;
    // the tiles' swizzle goes by address: dynamic shared memory starts on 1024 bytes
    // where a kernel has no other (two CTAs leave no room to round up)
    if (smem_u32(sm) & 1023) {
        if (threadIdx.x == 0)
            atomicExch(&g_tc_error, TC_ERR_TIMEOUT);
        return;
    }
    const int n = (int)min((int64_t)C, sq.len - t0);
    const int64_t tile = slot * a.H + h;
    const int tid = threadIdx.x, lane = tid & 31;
    const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int q = warp & 3, half = warp >> 2;
    uint64_t *bars = reinterpret_cast<uint64_t *>(sm + GBAR);
    uint64_t *in_full = bars, *one_full = bars + 1, *k_full = bars + 2, *c_full = bars + 3,
             *two_full = bars + 4;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(bars + 5);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(bars + 6);
    if (tid == 0) {
        for (int i = 0; i < 5; ++i)
            mbar_init(&bars[i], 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(tslot, UCOLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = *tslot;
    const uint32_t lanes = tm + ((uint32_t)(32 * q) << 16);
    const float *betas = reinterpret_cast<const float *>(sm + GTAB), *logs = betas + C,
                *lows = logs + C;

    if (tid == 0) {
        const int hq = h / a.q.hdiv, t = (int)(sq.bos + t0), row = (int)sq.row;
        mbar_arrive_expect_tx(in_full, 3 * 16384 + 2 * ETILE + STILE + 3 * C * 4);
        bulk_load(sm + GTAB, P.sc.tab + (tile * TABS + TBETA) * C, 3 * C * 4, in_full);
        bulk_load(sm + GS, P.sc.s + tile * STILE, STILE, in_full);
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            tma_load_4d(sm + GD + b * 16384, &P.mdo, in_full, 64 * b, h, t, row);
            bulk_load(sm + GD + b * 16384 + 8192, P.sc.r + tile * ETILE + b * 8192, 8192, in_full);
            tma_load_4d(sm + GQ + b * 16384, &P.mq, in_full, 64 * b, hq, t, row);
            tma_load_4d(sm + GQ + b * 16384 + 8192, &P.mk, in_full, 64 * b, hq, t, row);
        }
        bulk_load(sm + GE, P.sc.e + tile * ETILE, ETILE, in_full);
        bulk_prefetch(P.sc.k + tile * STILE, STILE);
    }
    __syncwarp();
    bool ok = warp_all(bwait(in_full, 0, abort_flag));
    if (a.cu && n < C) {    // another sequence's tokens: zeros
        const uint4 z = make_uint4(0, 0, 0, 0);
        for (int x = tid; x < (C - n) * 8; x += GRADS) {
            const int off = (n + x / 8) * 128 + (x % 8) * 16;
#pragma unroll
            for (int b = 0; b < 4; ++b)
                *reinterpret_cast<uint4 *>(sm + GQ + b * 8192 + off) = z;
            *reinterpret_cast<uint4 *>(sm + GD + off) = z;
            *reinterpret_cast<uint4 *>(sm + GD + 16384 + off) = z;
        }
        fence_proxy_async_smem();
    }
    __syncthreads();
    const uint32_t sb = smem_u32(sm);
    constexpr uint32_t id64 = idesc_bf16_f32(128, 64, 0, 0), id128 = idesc_bf16_f32(128, 128, 0, 1);
    if (warp == 0 && ok && elect_one()) {
        const uint64_t d_d = sdesc_sw128(sb + GD, 16, 1024), d_e = sdesc_sw128(sb + GE, 16, 1024);
        const uint64_t d_s = sdesc_sw128(sb + GS, 16384, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)      // [dO; R] Eps^T
            mma_ss(tm + UW, d_d + ((kk >> 2) * 1024 + (kk & 3) * 2),
                   d_e + ((kk >> 2) * 512 + (kk & 3) * 2), id64, kk > 0);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)      // [dO; R] S^T
            mma_ss(tm + U1, d_d + ((kk >> 2) * 1024 + (kk & 3) * 2), d_s + kk * 128, id128, kk > 0);
        mma_commit(one_full);
    }
    __syncwarp();
    // this thread's share of S for <S, K'>
    uint4 sv[8];
#pragma unroll
    for (int x = 0; x < 8; ++x)
        sv[x] = *reinterpret_cast<const uint4 *>(sm + GS + tid * 16 + x * 4096);
    ok = warp_all(bwait(one_full, 0, abort_flag)) && ok;
    tc_fence_after();
    __syncthreads();    // S has been read, by the products and by every thread
    if (tid == 0 && ok) {
        mbar_arrive_expect_tx(k_full, STILE);
        bulk_load(sm + GS, P.sc.k + tile * STILE, STILE, k_full);
    }
    __syncwarp();
    const int i = 32 * (q & 1) + lane;              // this lane's token
    const bool key = q >= 2;                        // R's lanes: dK's row part
    const float gi = logs[i], eg = exp2_fast(gi), beta = betas[i];
    const float li = lows[i];
    {   // W1 (W2), row i, columns 32 half .., as rows and as columns
        const int j0 = 32 * half;
        uint32_t r[32];
        tmem_ld32(lanes + UW + j0, r);
        if (key && i >= j0 && i < j0 + 32 && i < n) {
            float d = 0.f;
#pragma unroll
            for (int x = 0; x < 32; ++x)
                d = j0 + x == i ? __uint_as_float(r[x]) : d;
            static_cast<__nv_bfloat16 *>(a.dbeta)[((sq.row * a.T) + sq.bos + t0 + i) * a.H + h] =
                __float2bfloat16_rn(d);
        }
        const float f = key ? -beta : a.scale;
        const float2 f2 = make_float2(f, f), gi2 = make_float2(gi, gi), li2 = make_float2(li, li);
        const float2 minus = make_float2(-1.f, -1.f);
        const int last = key ? i - 1 : i;
        float w[32];
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            auto pair = [&](const float *t) {
                return *reinterpret_cast<const float2 *>(t + j0 + 2 * x);
            };
            const float2 d = add2(fma2(pair(logs), minus, gi2), fma2(pair(lows), minus, li2));
            const float2 y = mul2(mul2(mul2(f2, pair(betas)),
                                       make_float2(exp2_fast(d.x), exp2_fast(d.y))),
                                  pair_of(r, x));
            w[2 * x] = j0 + 2 * x <= last ? y.x : 0.f;
            w[2 * x + 1] = j0 + 2 * x + 1 <= last ? y.y : 0.f;
        }
        put_half_row(sm + GW + (key ? 8192 : 0) + i * 128, i, 4 * half, w);
        uint8_t *to = sm + GWT + (key ? 8192 : 0) + (i & 6) * 2;
        const bool odd = lane & 1;
#pragma unroll
        for (int m = 0; m < 16; ++m) {
            const float mine = odd ? w[2 * m + 1] : w[2 * m], other = odd ? w[2 * m] : w[2 * m + 1];
            const float got = __shfl_xor_sync(0xffffffffu, other, 1);
            const int j = j0 + 2 * m + odd;
            *reinterpret_cast<uint32_t *>(to + j * 128 + (((i >> 3) ^ (j & 7)) << 4)) =
                odd ? pack_bf16x2(got, mine) : pack_bf16x2(mine, got);
        }
    }
    {   // the products with S, scaled
        const float f = key ? -eg * beta : a.scale * eg;
        const float2 f2 = make_float2(f, f);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            uint32_t r[32];
            tmem_ld32(lanes + U1 + 64 * half + 32 * p, r);
#pragma unroll
            for (int x = 0; x < 16; ++x)
                put_pair(r, x, mul2(f2, pair_of(r, x)));
            tmem_st32_issue(lanes + U1 + 64 * half + 32 * p, r);
        }
        tmem_wait_st();
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    ok = warp_all(bwait(k_full, 0, abort_flag)) && ok;
    const bool issuer = warp == 0 && ok && elect_one();
    if (issuer) {
        const uint64_t d_e = sdesc_sw128(sb + GE - 8192, 16, 1024);
        const uint64_t d_s = sdesc_sw128(sb + GS, 16384, 1024);
        const uint64_t d_w = sdesc_sw128(sb + GW, 16, 1024);
        const uint64_t d_k = sdesc_sw128(sb + GQ + 8192, 16384, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)      // Eps K'^T
            mma_ss(tm + UC, d_e + ((kk >> 2) * 512 + (kk & 3) * 2), d_s + kk * 128, id128, kk > 0);
        mma_commit(c_full);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)      // [W1; W2] K
            mma_ss(tm + U1, d_w + kk * 2, d_k + kk * 128, id128, 1);
    }
    __syncwarp();
    float end = 0.f;    // <S', K'>
    if (ok) {
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const uint4 kv = *reinterpret_cast<const uint4 *>(sm + GS + tid * 16 + x * 4096);
            const uint32_t u[4] = {sv[x].x, sv[x].y, sv[x].z, sv[x].w};
            const uint32_t w[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                end = fmaf(bf16lo(u[y]), bf16lo(w[y]), end);
                end = fmaf(bf16hi(u[y]), bf16hi(w[y]), end);
            }
        }
        end *= exp2_fast(logs[C - 1]);
    }
    // row i of Q (K): this half's 64 channels
    const uint8_t *own = sm + GQ + half * 16384 + (key ? 8192 : 0) + i * 128;
    ok = warp_all(bwait(c_full, 0, abort_flag)) && ok;
    tc_fence_after();
    if (key) {
        const float f = beta * exp2_fast((logs[C - 1] - gi) + (lows[C - 1] - li));
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
            uint32_t r[32];
            float x32[32];
            tmem_ld32(lanes + UC + 64 * half + 32 * p, r);
#pragma unroll
            for (int x = 0; x < 32; ++x) {
                x32[x] = f * __uint_as_float(r[x]);
                r[x] = __float_as_uint(x32[x]);
            }
            tmem_st32_issue(lanes + UC + 64 * half + 32 * p, r);
            end += row_dot(own, i, 4 * p, x32);
        }
        tmem_wait_st();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (issuer) {
        const uint64_t d_wt = sdesc_sw128(sb + GWT - 8192, 16, 1024);
        const uint64_t d_q = sdesc_sw128(sb + GQ, 16384, 1024);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)      // [W1^T, W2^T] [Q; K]
            mma_ss(tm + UC, d_wt + ((kk >> 2) * 512 + (kk & 3) * 2), d_q + kk * 128, id128, 1);
        mma_commit(two_full);
    }
    __syncwarp();
    ok = warp_all(bwait(two_full, 0, abort_flag)) && ok;
    tc_fence_after();
    float *red = reinterpret_cast<float *>(sm + GS);        // [4][64], then 8 sums
    if (ok) {
        float t = 0.f;
        // dq (dk) of token i, 64 channels: out through the tile of Eps (of dO)
        uint8_t *stage = sm + (key ? GD : GE) + half * 8192 + i * 128;
        float *part = P.sc.dqp ? (key ? P.sc.dkp : P.sc.dqp) +
                                     ((sq.row * a.T + sq.bos + t0 + i) * a.H + h) * a.D + 64 * half
                               : nullptr;
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
            uint32_t r[32];
            float x32[32], y32[32];
            tmem_ld32(lanes + U1 + 64 * half + 32 * p, r);
#pragma unroll
            for (int x = 0; x < 32; ++x)
                x32[x] = y32[x] = __uint_as_float(r[x]);
            if (key) {
                tmem_ld32(lanes + UC + 64 * half + 32 * p, r);
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                    const float col = __uint_as_float(r[x]);
                    y32[x] = x32[x] - col;
                    x32[x] += col;
                }
            }
            t += row_dot(own, i, 4 * p, y32);
            if (!part)
                put_half_row(stage, i, 4 * p, x32);
            else if (i < n)
#pragma unroll
                for (int x = 0; x < 32; x += 4)
                    if (64 * half + 32 * p + x < a.D)
                        *reinterpret_cast<float4 *>(part + 32 * p + x) =
                            make_float4(x32[x], x32[x + 1], x32[x + 2], x32[x + 3]);
        }
        red[64 * (2 * (q >> 1) + half) + i] = t;
#pragma unroll
        for (int m = 1; m < 32; m *= 2)
            end += __shfl_xor_sync(0xffffffffu, end, m);
        if (lane == 0)
            red[256 + warp] = end;
    }
    if (tid == 0 && !ok) {  // a wait ran out: what is in flight ends before the CTA does
        drain_wait(in_full, 0);
        drain_wait(one_full, 0);
        drain_wait(k_full, 0);
        drain_wait(c_full, 0);
        drain_wait(two_full, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0)
        tmem_dealloc(tm, UCOLS);
    if (!P.sc.dqp && ok)
#pragma unroll
        for (int x = 0; x < 8; ++x) {
            const int j = ((tid >> 4) + 16 * x) & 63, c16 = tid & 15;
            const TokOut &o = x < 4 ? a.dq : a.dk;
            if (j < n && 8 * c16 < a.D)
                *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(o.p) + sq.row * o.sb +
                                           (sq.bos + t0 + j) * o.st + (int64_t)h * o.sh +
                                           8 * c16) =
                    *reinterpret_cast<const uint4 *>(sm + (x < 4 ? GE : GD) + (c16 >> 3) * 8192 +
                                                     j * 128 + (((c16 & 7) ^ (j & 7)) << 4));
        }
    if (warp == 7) {    // dg: running sums from the chunk's last token
        float run = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w)
            run += red[256 + w];
#pragma unroll
        for (int p = 1; p >= 0; --p) {
            const int j = 32 * p + 31 - lane;
            float x = red[j] + red[64 + j] + red[128 + j] + red[192 + j];
#pragma unroll
            for (int m = 1; m < 32; m *= 2) {
                const float y = __shfl_up_sync(0xffffffffu, x, m);
                if (lane >= m)
                    x += y;
            }
            if (j < n && ok)
                static_cast<__nv_bfloat16 *>(a.dg)[((sq.row * a.T) + sq.bos + t0 + j) * a.H + h] =
                    __float2bfloat16_rn(run + x);
            run += __shfl_sync(0xffffffffu, x, 31);
        }
    }
}

// ---- scan over segments -------------------------------------------------------------
//
// The states that enter a sequence's segments: S_0 the initial state, S_j+1 = Phi_j S_j +
// H_j; back K'_last = dL/dfinal, K'_j-1 = Phi_j^T K'_j + H_j.  A CTA takes 8 columns of a
// (sequence, head)'s state, two threads a row, in fp32; the next Phi is on its way into
// shared memory meanwhile.  Its steps are one after another: 128 x 128 x 8 products each.
constexpr int SCAN_COLS = 8, SCAN = 256;
constexpr int PP = 132;         // floats a row of Phi: neighbouring rows, other banks
constexpr int SCAN_DYN = (2 * 128 * PP + 2 * 128 * SCAN_COLS) * 4;
template <bool BWD>
__global__ void __launch_bounds__(SCAN) delta_scan_kernel(const DeltaArgs a, const Scratch sc,
                                                          int segs, int seg_len)
{
    extern __shared__ __align__(16) float scan_sm[];
    float *M[2] = {scan_sm, scan_sm + 128 * PP};
    float(*S)[128][SCAN_COLS] = reinterpret_cast<float(*)[128][SCAN_COLS]>(scan_sm + 2 * 128 * PP);
    const int cols = (a.E + SCAN_COLS - 1) / SCAN_COLS;
    const int h = blockIdx.x / cols % a.H, n = blockIdx.x / cols / a.H;
    const int c0 = 4 * (threadIdx.x & 1), d = threadIdx.x >> 1;
    const int e0 = blockIdx.x % cols * SCAN_COLS + c0;
    const Seq sq = sequence(a.cu, a.T, n);
    // never more than there is room for, whatever the table on the device says
    const int count = sq.len > 0 ? (int)min((sq.len + seg_len - 1) / seg_len, (int64_t)segs) : 1;
    const bool row = d < a.D;
    auto at = [&](int i) {      // the i-th segment in the scan's order
        return ((int64_t)n * segs + (BWD ? count - 1 - i : i)) * a.H + h;
    };
    auto ask = [&](int i) {
        if (i < count - 1) {
            const float *from = sc.phi + at(i) * a.D * a.D;
            for (int u = threadIdx.x; u < a.D * a.D / 4; u += SCAN) {
                const int r = u / (a.D / 4), c = 4 * (u - r * (a.D / 4));
                asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                 smem_u32(M[i & 1] + r * PP + c)),
                             "l"(from + r * a.D + c)
                             : "memory");
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    ask(0);
    const float *first = BWD ? a.dfin : a.init;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);     // E is a multiple of 8
    if (first && row) {
        first += (((int64_t)n * a.H + h) * a.D + d) * a.E + e0;
        x = make_float4(first[0], first[1], first[2], first[3]);
    }
    for (int i = 0;; ++i) {
        if (row)
            *reinterpret_cast<float4 *>(sc.enter + (at(i) * a.D + d) * a.E + e0) = x;
        if (i == count - 1)
            return;
        ask(i + 1);
        *reinterpret_cast<float4 *>(&S[i & 1][d][c0]) = x;
        if (row)
            x = *reinterpret_cast<const float4 *>(sc.own + (at(i) * a.D + d) * a.E + e0);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        __syncthreads();
        if (row) {
            const float *m = M[i & 1] + (BWD ? d : d * PP);
#pragma unroll 4
            for (int k = 0; k < a.D; k += 4) {      // D is a multiple of 8
                float f[4];
                if (BWD) {
#pragma unroll
                    for (int y = 0; y < 4; ++y)
                        f[y] = m[(k + y) * PP];
                } else {
                    const float4 v = *reinterpret_cast<const float4 *>(m + k);
                    f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
                }
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const float4 s = *reinterpret_cast<const float4 *>(&S[i & 1][k + y][c0]);
                    x.x = fmaf(f[y], s.x, x.x);
                    x.y = fmaf(f[y], s.y, x.y);
                    x.z = fmaf(f[y], s.z, x.z);
                    x.w = fmaf(f[y], s.w, x.w);
                }
            }
        }
        __syncthreads();        // M[i & 1] is asked for again in the next round
    }
}

// ---- host -------------------------------------------------------------------------

// Segments of a sequence: the count with the least time by this model, of a chunk's time
// in a sweep of states (2.6 us) and in one with outputs (3.2), rounds of CTAs on a GB300's
// 152 SMs, and 4 us a step of the scan with its launches.  The times are those of 128 x
// 128; narrower states take less in the scan alone.  Forward, one sequence, us, whole and
// in the segments taken (D = E = 128; 64):
//     1 head n2048     131, 80;      130, 66        1 head n65536    3570, 328;   3560, 258
//     16 heads n2047   134, 104;     131, 81        16 heads n65536  3730, 1350;  3710, 1220
//     32 heads n4096   266, 224;     261, 195       32 heads n32768  1980, 1330;  1960, 1220
// and where it stays whole (the best count, forced): 1 head n1024 74 (68; 54), 48 heads
// n16384 1050 (984; 940), 76 heads n16384 1150 (1110; 1056), 128 heads n16384 1330 (2100).
// The query of the sizes is a host function, so the SMs are not asked of the device.
struct Segments {
    int count, tokens;
};
Segments segments_of(const DeltaArgs &a)
{
    const int64_t pairs = (int64_t)a.N * a.H, chunks = (a.longest + C - 1) / C;
    const int64_t sms = 152;
    Segments best{1, (int)(chunks * C)};
    if (pairs == 0 || pairs > sms / 2)
        return best;
    double least = 0.9 * 3.2 * (double)chunks;      // a split has to be worth it
    for (int64_t n = 2; n <= 64 && 4 * n <= chunks; ++n) {
        const int64_t len = (chunks + n - 1) / n, count = (chunks + len - 1) / len;
        const int64_t first = (2 * pairs * (count - 1) + sms - 1) / sms;
        const int64_t second = (pairs * count + sms - 1) / sms;
        const double t = (2.6 * (double)first + 3.2 * (double)second) * (double)len +
                         4.0 * (double)count + 10.0;
        if (t < least) {
            least = t;
            best = Segments{(int)count, (int)(len * C)};
        }
    }
    return best;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }
size_t tiles_of(const DeltaArgs &a)
{
    return (size_t)slots_of(a.N, a.T, a.cu != nullptr) * a.H;
}
size_t prep_bytes(const DeltaArgs &a) { return tiles_of(a) * (BTILE + TAB); }

// Phi, and the states of segments (each of two buffers); 0 for whole sequences
size_t phi_bytes(const DeltaArgs &a)
{
    const int n = segments_of(a).count;
    return n > 1 ? up((size_t)a.N * n * a.H * a.D * a.D * sizeof(float)) : 0;
}
size_t segment_bytes(const DeltaArgs &a)
{
    const int n = segments_of(a).count;
    return n > 1 ? up((size_t)a.N * n * a.H * a.D * a.E * sizeof(float)) : 0;
}
void put_segments(const DeltaArgs &a, uint8_t *p, Scratch *sc)
{
    sc->own = reinterpret_cast<float *>(p);
    sc->enter = reinterpret_cast<float *>(p + segment_bytes(a));
}

void put_saved(const DeltaArgs &a, uint8_t *p, bool keep, Scratch *sc)
{
    const size_t t = tiles_of(a);
    sc->phi = reinterpret_cast<float *>(
        p + up(prep_bytes(a) + (keep ? t * (STILE + ETILE) : 0)));
    sc->b = p;
    sc->tab = reinterpret_cast<float *>(p + t * BTILE);
    sc->s = keep ? p + prep_bytes(a) : nullptr;
    sc->e = keep ? sc->s + t * STILE : nullptr;
}

bool token_map(CUtensorMap *m, const DeltaArgs &a, const Tok &x, int heads, int width)
{
    SweepArgs s{};
    s.B = a.B;
    s.T = a.T;
    s.H = heads;
    return make_map(m, x.p, width, s, x.sb, x.st, x.sh, C);
}

template <bool BWD> cudaError_t sweep(const DeltaArgs &a, const Scratch &sc, cudaStream_t s)
{
    SweepParams p;
    if (!token_map(&p.mq, a, a.q, a.HK, a.D) || !token_map(&p.mk, a, a.k, a.HK, a.D) ||
        !token_map(&p.mv, a, BWD ? a.d_o : a.v, a.H, a.E))
        return cudaErrorNotSupported;
    const TokOut &out = BWD ? a.dv : a.o;
    if (out.p && !token_map(&p.mo, a, Tok{out.p, out.sb, out.st, out.sh, 1}, a.H, a.E))
        return cudaErrorNotSupported;
    p.a = a;
    p.sc = sc;
    const Segments seg = segments_of(a);
    p.segs = seg.count;
    p.seg_len = seg.tokens;
    p.states = 0;
    cudaError_t e = cudaFuncSetAttribute(delta_sweep_kernel<BWD>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         SweepLayout<BWD>::DYN);
    if (e != cudaSuccess)
        return e;
    const unsigned ctas = (unsigned)((int64_t)a.N * seg.count * a.H);
    if (seg.count > 1) {
        SweepParams first = p;
        first.states = 1;
        delta_sweep_kernel<BWD>
            <<<dim3(ctas, BWD ? 1 : 2), SWEEP, SweepLayout<BWD>::DYN, s>>>(first);
        note_launch();
        if ((e = cudaGetLastError()) != cudaSuccess)
            return e;
        const unsigned cols = (unsigned)((a.E + SCAN_COLS - 1) / SCAN_COLS);
        e = cudaFuncSetAttribute(delta_scan_kernel<BWD>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, SCAN_DYN);
        if (e != cudaSuccess)
            return e;
        delta_scan_kernel<BWD>
            <<<(unsigned)(a.N * a.H) * cols, SCAN, SCAN_DYN, s>>>(a, sc, seg.count, seg.tokens);
        note_launch();
        if ((e = cudaGetLastError()) != cudaSuccess)
            return e;
        p.a.withhold_handoff = 0;
    }
    delta_sweep_kernel<BWD><<<ctas, SWEEP, SweepLayout<BWD>::DYN, s>>>(p);
    note_launch();
    return cudaGetLastError();
}

}  // namespace

bool delta_tc_row_ok(const void *p, const int64_t *st, int B, int T, int heads)
{
    const int n[3] = {B, T, heads};
    for (int i = 0; i < 3; ++i)
        if (n[i] > 1 && (st[i] <= 0 || st[i] % 8))
            return false;
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

bool delta_tc_sized(const DeltaArgs &a)
{
    if (!a.bf16 || a.D % 8 || a.E % 8 || a.D > 128 || a.E > 128 || a.longest <= SHORT_MAX_T)
        return false;
    const Tok *t[3] = {&a.q, &a.k, &a.v};
    for (int i = 0; i < 3; ++i) {
        const int64_t st[3] = {t[i]->sb, t[i]->st, t[i]->sh};
        if (!delta_tc_row_ok(nullptr, st, a.B, a.T, i < 2 ? a.HK : a.H))
            return false;
    }
    return tiles_of(a) <= INT_MAX;
}

size_t delta_tc_saved_bytes(const DeltaArgs &a)
{
    return up(prep_bytes(a) + tiles_of(a) * (STILE + ETILE)) + phi_bytes(a);
}

size_t delta_tc_fwd_bytes(const DeltaArgs &a, bool keep)
{
    return 2 * segment_bytes(a) + (keep ? 0 : up(prep_bytes(a)) + phi_bytes(a));
}

size_t delta_tc_bwd_bytes(const DeltaArgs &a)
{
    const size_t parts = a.H == a.HK ? 0 : up((size_t)a.B * a.T * a.H * a.D * sizeof(float));
    return up(tiles_of(a) * (STILE + ETILE)) + 2 * parts + 2 * segment_bytes(a);
}

cudaError_t delta_tc_forward(const DeltaArgs &a, cudaStream_t s)
{
    if (a.N == 0)
        return cudaSuccess;
    Scratch sc{};
    // the workspace: the segments' states, then what is not saved
    put_segments(a, a.ws, &sc);
    put_saved(a, a.saved ? a.saved : a.ws + 2 * segment_bytes(a), a.saved != nullptr, &sc);
    delta_prep_kernel<<<(unsigned)tiles_of(a), PREP, 0, s>>>(a, sc);
    note_launch();
    const cudaError_t e = cudaGetLastError();
    return e != cudaSuccess ? e : sweep<false>(a, sc, s);
}

cudaError_t delta_tc_backward(const DeltaArgs &a, cudaStream_t s)
{
    if (a.N == 0)
        return cudaSuccess;
    Scratch sc{};
    const size_t t = tiles_of(a);
    put_saved(a, a.saved, true, &sc);
    sc.k = a.ws;
    sc.r = a.ws + t * STILE;
    const size_t images = up(t * (STILE + ETILE));
    put_segments(a, a.ws + images, &sc);
    if (a.H != a.HK) {
        const size_t parts = up((size_t)a.B * a.T * a.H * a.D * sizeof(float));
        uint8_t *at = a.ws + images + 2 * segment_bytes(a);
        sc.dqp = reinterpret_cast<float *>(at);
        sc.dkp = reinterpret_cast<float *>(at + parts);
    }
    cudaError_t e = sweep<true>(a, sc, s);
    if (e != cudaSuccess)
        return e;
    GradParams p;
    if (!token_map(&p.mq, a, a.q, a.HK, a.D) || !token_map(&p.mk, a, a.k, a.HK, a.D) ||
        !token_map(&p.mdo, a, a.d_o, a.H, a.E))
        return cudaErrorNotSupported;
    p.a = a;
    p.sc = sc;
    e = cudaFuncSetAttribute(delta_grads_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, GDYN);
    if (e != cudaSuccess)
        return e;
    delta_grads_kernel<<<(unsigned)t, GRADS, GDYN, s>>>(p);
    note_launch();
    if ((e = cudaGetLastError()) != cudaSuccess || a.H == a.HK)
        return e;
    // a shared head's gradients: the sum over its group, fp32
    e = gqa_reduce(sc.dqp, a.dq, a.B, a.T, a.HK, a.H / a.HK, a.D, 1, s, true);
    return e != cudaSuccess ? e
                            : gqa_reduce(sc.dkp, a.dk, a.B, a.T, a.HK, a.H / a.HK, a.D, 1, s, true);
}

cudaError_t delta_read_and_clear_error(cudaStream_t s, int *err)
{
    return read_and_clear_error_word(s, err);
}

}  // namespace la
