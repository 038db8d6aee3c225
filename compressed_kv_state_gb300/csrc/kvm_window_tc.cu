// Sliding-window attention with sink tokens, forward, on the 5th-generation tensor
// cores (tcgen05 + TMEM + TMA).  bf16.
//
//   s_ij = q'_i . k'_j / 8 for j <= i and (i - j < W or j < S), out_i = softmax(s_i) v
//
// Work unit: 128 consecutive queries of one (b, h).  Its keys come in one sink block
// (keys [0, S), S rounded up to 16 columns) when some query's window starts past key 0,
// then blocks of 128 from the first key that any of its windows sees: with W = 512 five
// blocks and the narrow one, of which the first and the last are masked per row.
//
// Persistent CTAs (one per SM, 384 threads, 225 KB shared memory, all 512 tensor-memory
// columns) hold two tiles in flight, each with roles of its own, so that the tensor core
// runs one tile's products while the other's softmax works:
//   warps 0, 1    producers: Q tile, K and V blocks (three stages each) by TMA
//   warps 2, 3    one thread issues S = Q K^T, then O += P V with P read from tensor
//                 memory; the next block's S goes out before this block's P is ready
//   warps 4-11    softmax: thread i owns query row i (= tensor-memory lane i): maximum,
//                 exponentials, lazy rescaling of O (only when the running maximum grows
//                 by more than 2^8, which fp32 sums absorb), P as bf16 pairs
// The softmax warps set the pace: B8 H12 N8192 W512 without rotation 213 us, no unit near a
// limit (tensor pipe 24%, exponentials 22%, issue 43%).  Three tiles of 64-key blocks in flight
// need them at 128 registers and then spill much more than the 80 bytes of this form (twice the
// time).
// Queries and keys are rotated by a pass before (of 32 rotary dims it stores just those,
// and a tile is then two half-row tiles, the second from the input itself); rotating the
// queries here, in warps of their own, slowed the softmax by more than the pass takes.
//
// A product with P reads whole blocks, and 0 x NaN is NaN: a row whose result is not
// finite is looked at again (repair_rows), so values behind the mask never reach it.
//
// All mbarrier waits are bounded (about two seconds); on expiry the CTA raises the
// status word, lets its copies and MMAs land, and exits.
#include <cuda.h>

#include "kvm_window.cuh"
#include "tc_primitives.cuh"

namespace kvm {
namespace wint {

using namespace tc;

constexpr int NSLOT = 2;              // query tiles in flight
constexpr int NS = 3;                 // K stages and V stages per slot
constexpr int KB = 128;               // keys per block
constexpr int Q_BYTES = 128 * 128;    // [128][64] bf16, 128-byte swizzled rows
constexpr int KV_BYTES = KB * 128;
constexpr int OFF_Q = 0;
constexpr int OFF_K = OFF_Q + NSLOT * Q_BYTES;
constexpr int OFF_V = OFF_K + NSLOT * NS * KV_BYTES;
constexpr int OFF_BAR = OFF_V + NSLOT * NS * KV_BYTES;
constexpr int SMEM_BYTES = OFF_BAR + 512 + 1024;
constexpr int TMEM_COLS = 512, TMEM_SLOT = 256;  // of a slot: S (128), O (64), P (64: bf16 key pairs)
constexpr int NTHREADS = 384;
// launched with 168 registers a thread (64512): 128 x 64 + 256 x 216 = 63488
constexpr int REGS_LOW = 64, REGS_HIGH = 216;
constexpr float LOWEST = -3.4028234663852886e38f;
constexpr float TAU = 8.0f;  // lazy-rescale threshold (log2 units)

enum {
    B_QFULL = 0,               // TMA Q landed
    B_QEMPTY,                  // last S of the tile done
    B_KFULL,                   // [NS]
    B_KEMPTY = B_KFULL + NS,   // [NS] S of the stage done (last block: the output tile staged there has left)
    B_VFULL = B_KEMPTY + NS,   // [NS]
    B_VEMPTY = B_VFULL + NS,   // [NS] PV of the stage done
    B_SFULL = B_VEMPTY + NS,   // S done
    B_SFREE,                   // S read into registers (128 arrivals)
    B_PFULL,                   // P written, O rescaled (128 arrivals)
    B_PVDONE,                  // PV done
    B_OUT,                     // output tile in shared memory (128 arrivals)
    B_FINAL,                   // MMA drain
    NBAR
};

struct TcArgs {
    int N, H, W, S, SW, half;     // SW: columns of a sink block, S rounded up to 16, at most 128
    int ntiles, qtiles;
    FastDiv by_bh, by_h, by_g;    // B * H, H, H / Hkv
    Rows q, k, v;                 // q, k as the scores use them (rotated; with split, dims [0, 32) alone)
    Rows q_in, k_in;              // split: the unrotated ones, read for dims [32, 64)
    int split;
    float* lse;
    float scale_log2;
    int* status;
};

struct Tile {
    int b, h, hk, sink, nblk;
    int q0, ws;
};

// Tiles are numbered from the last queries back: with a long window those are the
// largest, and the persistent CTAs then end with small ones.
__device__ __forceinline__ Tile tile_of(const TcArgs& a, int id) {
    Tile t;
    const int qb = a.by_bh.div(id), bh = id - qb * (int)a.by_bh.d;
    t.b = a.by_h.div(bh);
    t.h = bh - t.b * a.H;
    t.hk = a.by_g.div(t.h);
    t.q0 = (a.qtiles - 1 - qb) * 128;
    const int q1 = min(t.q0 + 128, a.N);
    t.ws = max(t.q0 - a.W + 1, 0);
    // the sinks are blocks of their own once the tile's last query does not see key 0 otherwise
    t.sink = a.S > 0 && q1 > a.W ? (a.S + KB - 1) / KB : 0;
    if (t.sink) t.ws = max(t.ws, a.S);
    t.nblk = t.sink + (t.ws < q1 ? (q1 - t.ws + KB - 1) / KB : 0);
    return t;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}

// bounded wait with no abort shortcut (drains after an abort)
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try(bar, parity) && clock64() - t0 < (1ll << 28)) {
    }
}

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ bool odd(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

// s[y] of a lane becomes its own and lane ^ W's s[y] or, in the upper of the two, s[y + W]
template <int W> __device__ __forceinline__ void halve(float (&s)[32], int lane) {
#pragma unroll
    for (int y = 0; y < W; ++y) {
        const float give = lane & W ? s[y] : s[y + W], have = lane & W ? s[y + W] : s[y];
        s[y] = have + __shfl_xor_sync(0xffffffffu, give, W);
    }
}

// Rows of a warp whose results are not finite, by the whole warp: bit r of `rows` is query p0 + r,
// whose maximum and sum of weights are lane r's m and l, whose result is row r at `out`.
//
// Such a result is right where a key that the row sees is to blame.  But a product multiplies
// whole blocks and 0 x NaN is NaN, so it may also be a value of a key in the tile's blocks that
// the row does not see.  Those are few, at most 127 before the window of the warp's last row and
// 254 behind its first, and are looked at first.  Dims that such a value reaches are computed
// again from the keys that the row does see, until none of them can become finite any more; at
// most 381 rows of a head come this far for one such value.  Four rows and eight keys at a time,
// two dims a lane: 1,700 cycles (a NaN in every head of B1 H2 N16384, causal: 190 us where every
// later row sees it, 7.6 ms where 127 rows of a tile do not).  Meanwhile `work` is counted up, so
// that the CTA's waits last.
__device__ __noinline__ void repair_rows(const TcArgs& a, const Tile& T, int p0, uint32_t rows, float m, float l, uint8_t* out,
                                         volatile int* work) {
    constexpr uint32_t ALL = 0xffffffffu;
    const int lane = threadIdx.x & 31;
    auto below = [](int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; };
    auto word = [&](const Rows& x, int h, int j, int w) { return reinterpret_cast<const uint32_t*>(x.at<const __nv_bfloat16>(T.b, h, j))[w]; };
    const Rows &qr = a.split && lane >= 16 ? a.q_in : a.q, &kr = a.split && lane >= 16 ? a.k_in : a.k;
    // bit r: dim 2 lane (bad0) or 2 lane + 1 (bad1) of row r is reached by a key out of its sight
    uint32_t bad0 = 0, bad1 = 0;
    auto look = [&](int j, int end) {
#pragma unroll 8
        for (; j < end; ++j) {
            const uint32_t w = word(a.v, T.hk, j, lane), blind = below(j - p0) | (j >= a.S ? ~below(j + a.W - p0) : 0);
            if (odd(lo_f(w))) bad0 |= blind;
            if (odd(hi_f(w))) bad1 |= blind;
        }
    };
    const int end = min(T.ws + KB * (T.nblk - T.sink), a.N);
    if (T.sink) look(p0 + 1, a.S);  // (rows past the sinks' are zeros in their block)
    look(T.ws, min(p0 + 32 - a.W, min(p0 + 1, end)));
    look(max(p0 + 1, T.ws), end);
    rows &= __reduce_or_sync(ALL, bad0 | bad1);
    __syncwarp();  // (each row has been stored by its own lane)
    while (rows) {
        int r[4], p[4];  // (p -1: no row)
        float q0[4], q1[4], o0[4], o1[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            r[x] = rows ? __ffs(rows) - 1 : 0;
            p[x] = rows ? p0 + r[x] : -1;
            rows &= rows - 1;
            const uint32_t w = p[x] >= 0 ? word(qr, T.h, p[x], lane) : 0;
            q0[x] = lo_f(w);
            q1[x] = hi_f(w);
            o0[x] = o1[x] = 0.f;
        }
        const int px = p[0] < 0 ? -1 : lane < 8 ? p[0] : lane < 16 ? p[1] : lane < 24 ? p[2] : p[3];  // of this lane's score
        const float mx = __shfl_sync(ALL, m, lane < 8 ? r[0] : lane < 16 ? r[1] : lane < 24 ? r[2] : r[3]);
        const int last = max(max(p[0], p[1]), max(p[2], p[3])), ws = max(p[0] - a.W + 1, 0), sinks = min(a.S, ws);
        const int chunks = (sinks + 7) / 8, n = chunks + (last - ws) / 8 + 1;  // of eight keys: sinks, then from ws on
        uint32_t kw[8], vw[8];
        auto fetch = [&](int i) {
            const int j0 = i < chunks ? 8 * i : ws + 8 * (i - chunks);
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int j = min(j0 + u, a.N - 1);
                kw[u] = word(kr, T.hk, j, lane);
                vw[u] = word(a.v, T.hk, j, lane);
            }
        };
        fetch(0);
        for (int i = 0; i < n; ++i) {
            float s[32];
#pragma unroll
            for (int u = 0; u < 8; ++u)
#pragma unroll
                for (int x = 0; x < 4; ++x) s[8 * x + u] = fmaf(q1[x], hi_f(kw[u]), q0[x] * lo_f(kw[u]));
            uint32_t v[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) v[u] = vw[u];
            if (i + 1 < n) fetch(i + 1);
            // lane 8 x + u ends with the sum of row x and key u over the lanes
            halve<16>(s, lane);
            halve<8>(s, lane);
            halve<4>(s, lane);
            halve<2>(s, lane);
            halve<1>(s, lane);
            const int j = (i < chunks ? 8 * i : ws + 8 * (i - chunks)) + (lane & 7);
            const bool seen = (i >= chunks || j < sinks) && j <= px && (px - j < a.W || j < a.S);
            const float e = seen ? ex2(fmaf(s[0], a.scale_log2, -mx)) : -0.f;  // (a weight is never -0)
#pragma unroll
            for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const float w = __shfl_sync(ALL, e, 8 * x + u);
                    const bool skip = __float_as_uint(w) == 0x80000000u;
                    o0[x] = skip ? o0[x] : fmaf(w, lo_f(v[u]), o0[x]);
                    o1[x] = skip ? o1[x] : fmaf(w, hi_f(v[u]), o1[x]);
                }
            if ((i & 63) == 63) {
                bool may = false;
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    may = may || (p[x] >= 0 && (((bad0 >> r[x] & 1) && !odd(o0[x])) || ((bad1 >> r[x] & 1) && !odd(o1[x]))));
                if (!__any_sync(ALL, may)) break;
                if (lane == 0) *work = *work + 1;
            }
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float il = 1.f / __shfl_sync(ALL, l, r[x]);
            __nv_bfloat16* y = reinterpret_cast<__nv_bfloat16*>(out + r[x] * 128 + ((((lane >> 2) ^ (r[x] & 7)) << 4) | ((lane & 3) << 2)));
            if (p[x] >= 0 && (bad0 >> r[x] & 1)) y[0] = __float2bfloat16_rn(o0[x] * il);
            if (p[x] >= 0 && (bad1 >> r[x] & 1)) y[1] = __float2bfloat16_rn(o1[x] * il);
        }
    }
}

__global__ void __launch_bounds__(NTHREADS, 1)
    win_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_sk,
                  const __grid_constant__ CUtensorMap tm_sv, const __grid_constant__ CUtensorMap tm_o,
                  const __grid_constant__ CUtensorMap tm_qh, const __grid_constant__ CUtensorMap tm_kh,
                  const __grid_constant__ CUtensorMap tm_skh, const __grid_constant__ TcArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NSLOT * NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* work = abort_flag + 1;  // (counted up by repair_rows)
    auto bar = [&](int slot, int i) { return smem_u32(bars + slot * NBAR + i); };
    // turn k of slot s is tile blockIdx.x + (NSLOT k + s) * gridDim.x
    auto tile_id = [&](int slot, int k) -> int {
        const int64_t id = blockIdx.x + (int64_t)(NSLOT * k + slot) * gridDim.x;
        return id < a.ntiles ? (int)id : -1;
    };

    if (tid == 0) {
        for (int s = 0; s < NSLOT; ++s) {
            for (int i = 0; i < NS; ++i) {
                mbar_init(bar(s, B_KFULL + i), 1);
                mbar_init(bar(s, B_KEMPTY + i), 1);
                mbar_init(bar(s, B_VFULL + i), 1);
                mbar_init(bar(s, B_VEMPTY + i), 1);
            }
            mbar_init(bar(s, B_QFULL), 1);
            mbar_init(bar(s, B_QEMPTY), 1);
            mbar_init(bar(s, B_SFULL), 1);
            mbar_init(bar(s, B_SFREE), 128);
            mbar_init(bar(s, B_PFULL), 128);
            mbar_init(bar(s, B_PVDONE), 1);
            mbar_init(bar(s, B_OUT), 128);
            mbar_init(bar(s, B_FINAL), 1);
        }
        *abort_flag = 0;
        *work = 0;
        fence_barrier_init();
        fence_proxy_async();
    }
    if (warp == 2) tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const uint32_t sbase = smem_u32(smem);
    if (warp < 4)
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_LOW));
    else
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_HIGH));

    if (warp < NSLOT) {
        // ------------------------------------------------------------ producer
        const int slot = warp;
        if (lane == 0) {
            int g = 0, last_q = -1, last_k = -1, last_v = -1;
            bool ok = true;
            if (a.half) asm volatile("griddepcontrol.wait;" ::: "memory");  // the rotated rows are there
            for (int k = 0; ok; ++k) {
                const int id = tile_id(slot, k);
                if (id < 0) break;
                const Tile T = tile_of(a, id);
                if (k >= 1 && !mbar_wait_idle(bar(slot, B_QEMPTY), (k - 1) & 1, abort_flag, a.status, work)) break;
                {
                    const uint32_t dq = sbase + OFF_Q + slot * Q_BYTES, full = bar(slot, B_QFULL);
                    mbar_expect_tx(full, Q_BYTES);
                    tma_load_4d(dq, &tm_q, 0, T.q0, T.h, T.b, full);
                    if (a.split) tma_load_4d(dq + Q_BYTES / 2, &tm_qh, 32, T.q0, T.h, T.b, full);
                    last_q = k;
                }
                for (int j = 0; j < T.nblk; ++j, ++g) {
                    const int st = g % NS;
                    const uint32_t dk = sbase + OFF_K + (slot * NS + st) * KV_BYTES;
                    const uint32_t dv = sbase + OFF_V + (slot * NS + st) * KV_BYTES;
                    const bool sink = j < T.sink;
                    const int key0 = sink ? KB * j : T.ws + KB * (j - T.sink);
                    const uint32_t bytes = sink ? (uint32_t)a.SW * 128 : (uint32_t)KV_BYTES;
                    if (g >= NS && !mbar_wait_idle(bar(slot, B_KEMPTY + st), (g / NS - 1) & 1, abort_flag, a.status, work)) { ok = false; break; }
                    mbar_expect_tx(bar(slot, B_KFULL + st), bytes);
                    tma_load_4d(dk, sink ? &tm_sk : &tm_k, 0, key0, T.hk, T.b, bar(slot, B_KFULL + st));
                    if (a.split)
                        tma_load_4d(dk + KV_BYTES / 2, sink ? &tm_skh : &tm_kh, 32, key0, T.hk, T.b, bar(slot, B_KFULL + st));
                    last_k = g;
                    if (g >= NS && !mbar_wait_idle(bar(slot, B_VEMPTY + st), (g / NS - 1) & 1, abort_flag, a.status, work)) { ok = false; break; }
                    mbar_expect_tx(bar(slot, B_VFULL + st), bytes);
                    tma_load_4d(dv, sink ? &tm_sv : &tm_v, 0, key0, T.hk, T.b, bar(slot, B_VFULL + st));
                    last_v = g;
                }
            }
            // after an abort: the copies issued last on every stage land before exit
            if (*abort_flag) {
                if (last_q >= 0) drain(bar(slot, B_QFULL), last_q & 1);
                for (int i = 0; i < NS; ++i) {
                    if (last_k - i >= 0) drain(bar(slot, B_KFULL + (last_k - i) % NS), ((last_k - i) / NS) & 1);
                    if (last_v - i >= 0) drain(bar(slot, B_VFULL + (last_v - i) % NS), ((last_v - i) / NS) & 1);
                }
            }
        }
    } else if (warp < 2 * NSLOT) {
        // ---------------------------------------------------------- MMA issuer
        const int slot = warp - NSLOT;
        const bool lead = elect_one();
        {
            const uint32_t idesc_qk = idesc_bf16(128, KB, 0, 0), idesc_qs = idesc_bf16(128, a.SW > 0 ? a.SW : 16, 0, 0);
            const uint32_t idesc_pv = idesc_bf16(128, 64, 0, 1);
            const uint32_t tS = tmem + TMEM_SLOT * slot, tO = tS + 128, tP = tS + 192;
            // shared-memory descriptors (address field in 16-byte units: a K-step of 32 bytes
            // adds 2, 16 rows of a block add 128)
            const uint64_t dq0 = a.split ? sdesc_sw64(sbase + OFF_Q + slot * Q_BYTES)
                                         : sdesc_sw128(sbase + OFF_Q + slot * Q_BYTES, 16, 1024);
            const uint64_t dk0 = a.split ? sdesc_sw64(sbase + OFF_K + slot * NS * KV_BYTES)
                                         : sdesc_sw128(sbase + OFF_K + slot * NS * KV_BYTES, 16, 1024);
            // K-steps 2, 3: the same row, or the second half-row tile
            const uint32_t k_hi = a.split ? KV_BYTES / 2 >> 4 : 4, q_hi = a.split ? Q_BYTES / 2 >> 4 : 4;
            const uint64_t dv0 = sdesc_sw128(sbase + OFF_V + slot * NS * KV_BYTES, KV_BYTES, 1024);
            int g = 0;
            bool ok = true;
            // S = Q K^T of block gb, once the softmax has read block gb - 1's S
            auto issue_qk = [&](int gb, bool sink, bool last) -> bool {
                const int st = gb % NS;
                if (gb > 0 && !mbar_wait_warp_idle(bar(slot, B_SFREE), (gb - 1) & 1, abort_flag, a.status, work)) return false;
                if (!mbar_wait_warp_idle(bar(slot, B_KFULL + st), (gb / NS) & 1, abort_flag, a.status, work)) return false;
                tc_fence_after();
                const uint64_t dk = dk0 + (uint64_t)(st * (KV_BYTES >> 4));
                if (lead) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks)
                        mma_bf16_ss(tS, dq0 + (ks >> 1) * q_hi + 2 * (ks & 1), dk + (ks >> 1) * k_hi + 2 * (ks & 1), sink ? idesc_qs : idesc_qk, ks > 0);
                    mma_commit(bar(slot, B_SFULL));
                    // the tile's last K stage holds its output tile next (the softmax frees it); the
                    // query tile is free
                    mma_commit(bar(slot, last ? B_QEMPTY : B_KEMPTY + st));
                }
                __syncwarp();
                return true;
            };
            for (int k = 0; ok; ++k) {
                const int id = tile_id(slot, k);
                if (id < 0) break;
                const Tile T = tile_of(a, id);
                if (!mbar_wait_warp_idle(bar(slot, B_QFULL), k & 1, abort_flag, a.status, work)) break;
                tc_fence_after();
                if (!issue_qk(g, T.sink > 0, T.nblk == 1)) break;
                for (int j = 0; j < T.nblk; ++j) {
                    const int gj = g + j, st = gj % NS;
                    if (j + 1 < T.nblk && !issue_qk(gj + 1, j + 1 < T.sink, j + 2 == T.nblk)) { ok = false; break; }
                    if (!mbar_wait_warp_idle(bar(slot, B_PFULL), gj & 1, abort_flag, a.status, work) ||
                        !mbar_wait_warp_idle(bar(slot, B_VFULL + st), (gj / NS) & 1, abort_flag, a.status, work)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    // O += P V: P (two keys per column) from tensor memory, V from shared
                    const uint64_t dv = dv0 + (uint64_t)(st * (KV_BYTES >> 4));
                    const int steps = j < T.sink ? a.SW / 16 : KB / 16;
                    if (lead) {
#pragma unroll
                        for (int ks = 0; ks < KB / 16; ++ks)
                            if (ks < steps) mma_bf16_ts(tO, tP + 8 * ks, dv + 128 * ks, idesc_pv, (j > 0 || ks > 0) ? 1u : 0u);
                        mma_commit(bar(slot, B_PVDONE));
                        mma_commit(bar(slot, B_VEMPTY + st));
                    }
                    __syncwarp();
                }
                g += T.nblk;
            }
            // every MMA this thread issued completes before the tensor memory is released
            if (lead) mma_commit(bar(slot, B_FINAL));
            drain(bar(slot, B_FINAL), 0);
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int slot = (warp - 4) >> 2;
        const int row = tid - 128 - 128 * slot;  // query row = tensor-memory lane
        const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + lane_base + TMEM_SLOT * slot, tO = tS + 128, tP = tS + 192;
        const float sc = a.scale_log2;
        const float2 sc2 = make_float2(sc, sc);
        int g = 0, held = -1;  // held: K stage that an output tile is being stored from
        bool ok = true;
        for (int k = 0; ok; ++k) {
            const int id = tile_id(slot, k);
            if (id < 0) break;
            const Tile T = tile_of(a, id);
            const int p = T.q0 + row;
            float m_used = LOWEST, l = 0.0f;  // (finite: scores of -infinity before any other get weights of 0)
            for (int j = 0; j < T.nblk; ++j) {
                const int gj = g + j;
                const bool sink = j < T.sink;
                const int key0 = sink ? KB * j : T.ws + KB * (j - T.sink);
                // columns [lo, hi) are keys that this query sees; lane 0's and lane 31's bounds
                // enclose the warp's
                auto cap = [](int x) { return max(0, min(x, KB)); };
                const int w0 = T.q0 + (row & ~31) - key0 + 1, top = sink ? min(a.S - key0, KB) : KB, off = sink ? KB : a.W;
                const int hi = min(cap(w0 + lane), top), lo = cap(w0 + lane - off) * !sink;
                const int hi_min = min(cap(w0), top), hi_max = min(cap(w0 + 31), top);
                const int lo_min = cap(w0 - off) * !sink, lo_max = cap(w0 + 31 - off) * !sink;
                const int groups = sink ? (a.SW + 31) / 32 : KB / 32;  // of 32 columns
                constexpr uint32_t ALL = (1u << (KB / 32)) - 1;
                if (!mbar_wait_warp_idle(bar(slot, B_SFULL), gj & 1, abort_flag, a.status, work)) { ok = false; break; }
                tc_fence_after();
                uint32_t v[KB / 32][32];
#pragma unroll
                for (int h = 0; h < KB / 32; ++h)
                    if (h < groups) tmem_ld32(tS + 32 * h, v[h]);
                tmem_wait_ld();
                // S is in registers: the next block's S may overwrite it
                tc_fence_before();
                mbar_arrive(bar(slot, B_SFREE));
                // a group of 32 columns that none of the warp's rows sees is left out, one that
                // all see whole needs no mask
                float mx0 = -INFINITY, mx1 = -INFINITY;
                auto maxima = [&](int h) {
#pragma unroll
                    for (int x = 0; x < 32; x += 4) {
                        mx0 = fmax3(mx0, __uint_as_float(v[h][x]), __uint_as_float(v[h][x + 1]));
                        mx1 = fmax3(mx1, __uint_as_float(v[h][x + 2]), __uint_as_float(v[h][x + 3]));
                    }
                };
                uint32_t live = ALL;
                if (hi_min == KB && lo_max == 0) {
#pragma unroll
                    for (int h = 0; h < KB / 32; ++h) maxima(h);
                } else {
                    live = 0;
#pragma unroll
                    for (int h = 0; h < KB / 32; ++h) {
                        if (h >= groups || 32 * h >= hi_max || 32 * h + 32 <= lo_min) continue;
                        live |= 1u << h;
                        if (32 * h + 32 > hi_min || 32 * h < lo_max) {
                            const int x1 = max(0, min(hi - 32 * h, 32)), x0 = max(0, min(lo - 32 * h, 32));
                            const uint32_t seen = (x1 < 32 ? (1u << x1) - 1 : ~0u) & ~(x0 < 32 ? (1u << x0) - 1 : ~0u);
#pragma unroll
                            for (int x = 0; x < 32; ++x)
                                if (!(seen & (1u << x))) v[h][x] = __float_as_uint(-INFINITY);
                        }
                        maxima(h);
                    }
                }
                const float mblk = fmaxf(mx0, mx1) * sc;
                bool rescale = false;
                float alpha = 1.0f;
                if (mblk > m_used) {
                    if (m_used == LOWEST) {
                        m_used = mblk;
                    } else if (mblk > m_used + TAU) {
                        alpha = ex2(m_used - mblk);
                        m_used = mblk;
                        rescale = true;
                    }
                }
                l *= alpha;
                // the previous block's PV has read P and updated O
                if (gj > 0 && !mbar_wait_warp_idle(bar(slot, B_PVDONE), (gj - 1) & 1, abort_flag, a.status, work)) { ok = false; break; }
                tc_fence_after();
                // tensor-memory loads and stores are warp-wide: the whole warp rescales when any
                // of its rows must (the others by 1)
                if (__any_sync(0xffffffffu, rescale)) {
                    uint32_t o[32];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        tmem_ld32(tO + h * 32, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
                        tmem_st32(tO + h * 32, o);
                    }
                }
                // p = 2^(s * scale - m), row sum, P as bf16 key pairs
                const float2 mneg = make_float2(-m_used, -m_used);
                float2 rs[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                make_float2(0.f, 0.f)};
                auto exps = [&](int h) {
                    uint32_t pk[16];
#pragma unroll
                    for (int x = 0; x < 32; x += 2) {
                        const float2 s2 = make_float2(__uint_as_float(v[h][x]), __uint_as_float(v[h][x + 1]));
                        const float2 t2 = __ffma2_rn(s2, sc2, mneg);
                        const float2 e2 = make_float2(ex2(t2.x), ex2(t2.y));
                        rs[(x >> 1) & 3] = __fadd2_rn(rs[(x >> 1) & 3], e2);
                        pk[x >> 1] = pack_bf16(e2.x, e2.y);
                    }
                    tmem_st16(tP + 16 * h, pk);
                };
                if (live == ALL) {  // (straight-line code: groups one by one measured 20% slower over whole blocks)
#pragma unroll
                    for (int h = 0; h < KB / 32; ++h) exps(h);
                } else {
#pragma unroll
                    for (int h = 0; h < KB / 32; ++h) {
                        if (h >= groups) continue;
                        if (live & (1u << h)) {
                            exps(h);
                        } else {
                            uint32_t zero[16];
#pragma unroll
                            for (int x = 0; x < 16; ++x) zero[x] = 0;
                            tmem_st16(tP + 16 * h, zero);
                        }
                    }
                }
                tmem_wait_st();
                l += ((rs[0].x + rs[0].y) + (rs[1].x + rs[1].y)) + ((rs[2].x + rs[2].y) + (rs[3].x + rs[3].y));
                tc_fence_before();
                mbar_arrive(bar(slot, B_PFULL));
                if (held >= 0 && row == 0) {  // the last tile's output has left its K stage
                    bulk_wait_read();
                    mbar_arrive(bar(slot, B_KEMPTY + held));
                    held = -1;
                }
                __syncwarp();
            }
            if (!ok) break;
            // epilogue: O / l (a query sees itself: l > 0) through the last block's K stage
            const int gl = g + T.nblk - 1, st = gl % NS;
            uint8_t* const tile = smem + OFF_K + (slot * NS + st) * KV_BYTES;
            if (!mbar_wait_warp_idle(bar(slot, B_PVDONE), gl & 1, abort_flag, a.status, work)) { ok = false; break; }
            tc_fence_after();
            const float il = 1.0f / l;
            const float2 il2 = make_float2(il, il);
            float2 sum = make_float2(0.f, 0.f);  // 0 x every value: not a number when one is not finite
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t o[32];
                tmem_ld32(tO + h * 32, o);
                tmem_wait_ld();
#pragma unroll
                for (int x = 0; x < 32; x += 8) {
                    uint32_t pk[4];
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float2 y = __fmul2_rn(make_float2(__uint_as_float(o[x + 2 * u]), __uint_as_float(o[x + 2 * u + 1])), il2);
                        sum = __ffma2_rn(y, make_float2(0.f, 0.f), sum);
                        pk[u] = pack_bf16(y.x, y.y);
                    }
                    *reinterpret_cast<uint4*>(tile + row * 128 + (((h * 4 + (x >> 3)) ^ (row & 7)) << 4)) =
                        make_uint4(pk[0], pk[1], pk[2], pk[3]);
                }
            }
            tc_fence_before();
            if (a.lse && p < a.N) a.lse[((int64_t)T.b * a.H + T.h) * a.N + p] = m_used + log2f(l);
            // (without a sum above 0 a score is no number, or all are -infinity: nor is any dim then)
            const uint32_t strange = __ballot_sync(0xffffffffu, !(sum.x + sum.y == 0.f) && p < a.N && l > 0.f);
            if (strange) repair_rows(a, T, T.q0 + (row & ~31), strange, m_used, l, tile + (row & ~31) * 128, work);
            fence_proxy_async();
            mbar_arrive(bar(slot, B_OUT));
            if (row == 0) {
                ok = mbar_wait_idle(bar(slot, B_OUT), k & 1, abort_flag, a.status, work);
                if (ok) tma_store_4d(&tm_o, smem_u32(tile), 0, T.q0, T.h, T.b);
                bulk_commit();
                held = st;
            }
            ok = __all_sync(0xffffffffu, ok);
            g += T.nblk;
        }
        if (row == 0) bulk_wait_all();
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// q and k turned at their own positions into [B, H, N, 64] of their own.  half a multiple
// of 8: a thread a position and a 16-byte piece with its partner (or two pieces to copy),
// for some heads one after the other, so that it reads the angles once.  compact (half =
// 16): the 32 rotated dims alone, [B, H, N, 32].  Else a thread a row.
struct RotArgs {
    Rows q, k;
    __nv_bfloat16 *qd, *kd;
    const float2* rope;
    int half, N, H, Hkv, per, groups, compact;  // per: heads of a thread
    FastDiv by_n, by_groups;  // N; groups of `per` heads
    int units;                // (b, group, position)
};
__global__ void __launch_bounds__(256) win_rotate_kernel(const __grid_constant__ RotArgs a) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int half = a.half, lp = (half & 7) ? 0 : a.compact ? 1 : 2;  // log2 of threads a unit
    const int64_t i = blockIdx.x * 256ll + threadIdx.x;
    if ((i >> lp) >= a.units) return;
    const int u = (int)(i >> lp), bg = a.by_n.div(u), n = u - bg * a.N;
    const int b = a.by_groups.div(bg), g = bg - b * a.groups, heads = a.H + a.Hkv;
    const int row = a.compact ? 32 : D, h0 = g * a.per, h1 = min(h0 + a.per, heads);
    const float2* cs_row = a.rope + (int64_t)n * half;
    const int part = (int)(i & ((1 << lp) - 1)), hc = half >> 3;
    float4 cs[4];
    if (!(half & 7) && part < hc) {
#pragma unroll
        for (int x = 0; x < 4; ++x) cs[x] = reinterpret_cast<const float4*>(cs_row)[4 * part + x];
    }
    // heads [f, e) of one of the two
    auto run = [&](const Rows& in, __nv_bfloat16* out, int H, int f, int e) {
        const __nv_bfloat16* s = in.at<const __nv_bfloat16>(b, f, n);
        __nv_bfloat16* d = out + (((int64_t)b * H + f) * a.N + n) * row;
        const int64_t ds = in.sh, dd = (int64_t)a.N * row;
        if (half & 7) {
            for (; f < e; ++f, s += ds, d += dd) {
                for (int x = 0; x < half; ++x) {
                    const float2 c = cs_row[x];
                    const float va = __bfloat162float(s[x]), vb = __bfloat162float(s[x + half]);
                    d[x] = __float2bfloat16_rn(va * c.x - vb * c.y);
                    d[x + half] = __float2bfloat16_rn(vb * c.x + va * c.y);
                }
                for (int x = 2 * half; x < D; ++x) d[x] = s[x];
            }
        } else if (part >= hc) {  // pieces [2 hc, 8): thread part copies 2 part and 2 part + 1
#pragma unroll 4
            for (; f < e; ++f, s += ds, d += dd) {
                const uint4 x = reinterpret_cast<const uint4*>(s)[2 * part], y = reinterpret_cast<const uint4*>(s)[2 * part + 1];
                reinterpret_cast<uint4*>(d)[2 * part] = x;
                reinterpret_cast<uint4*>(d)[2 * part + 1] = y;
            }
        } else {
#pragma unroll 4
            for (; f < e; ++f, s += ds, d += dd) {
                uint4 A = reinterpret_cast<const uint4*>(s)[part], B = reinterpret_cast<const uint4*>(s)[part + hc];
                __nv_bfloat162* a2 = reinterpret_cast<__nv_bfloat162*>(&A);
                __nv_bfloat162* b2 = reinterpret_cast<__nv_bfloat162*>(&B);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    const float2 y = __bfloat1622float2(a2[x]), z = __bfloat1622float2(b2[x]);
                    a2[x] = __floats2bfloat162_rn(y.x * cs[x].x - z.x * cs[x].y, y.y * cs[x].z - z.y * cs[x].w);
                    b2[x] = __floats2bfloat162_rn(z.x * cs[x].x + y.x * cs[x].y, z.y * cs[x].z + y.y * cs[x].w);
                }
                reinterpret_cast<uint4*>(d)[part] = A;
                reinterpret_cast<uint4*>(d)[part + hc] = B;
            }
        }
    };
    run(a.q, a.qd, a.H, min(h0, a.H), min(h1, a.H));
    run(a.k, a.kd, a.Hkv, max(h0 - a.H, 0), max(h1 - a.H, 0));
}

}  // namespace wint

cudaError_t launch_win_rotate(const WinArgs& a, void* q, void* k, bool compact, cudaStream_t s) {
    using namespace wint;
    RotArgs r{};
    r.q = a.q;
    r.k = a.k;
    r.qd = static_cast<__nv_bfloat16*>(q);
    r.kd = static_cast<__nv_bfloat16*>(k);
    r.rope = a.rope;
    r.half = a.r / 2;
    r.N = (int)a.N;
    r.H = a.H;
    r.Hkv = a.Hkv;
    const bool vec = r.half % 8 == 0;
    // eight heads a thread once that leaves every SM two thousand threads
    r.per = vec && a.B * a.N * (a.H + a.Hkv) / 8 * 2 >= 152 * 2048 ? 8 : 1;
    r.groups = (a.H + a.Hkv + r.per - 1) / r.per;
    r.compact = compact;
    r.by_n = FastDiv((uint32_t)a.N);
    r.by_groups = FastDiv((uint32_t)r.groups);
    r.units = (int)(a.B * r.groups * a.N);  // (fits: check_window)
    const int64_t threads = (int64_t)r.units << (vec ? (compact ? 1 : 2) : 0);
    win_rotate_kernel<<<(unsigned)((threads + 255) / 256), 256, 0, s>>>(r);
    return cudaGetLastError();
}

size_t win_fwd_q_bytes(const WinArgs& a) {
    return a.r ? ((size_t)a.B * a.H * a.N * (a.r == 32 ? 32 : D) * 2 + 255) / 256 * 256 : 0;
}
size_t win_fwd_scratch(const WinArgs& a) {
    return a.r ? win_fwd_q_bytes(a) + (size_t)a.B * a.Hkv * a.N * (a.r == 32 ? 32 : D) * 2 : 0;
}

cudaError_t launch_win_fwd_tc(const WinArgs& a, void* scratch, cudaStream_t s) {
    using namespace wint;
    TcArgs t{};
    t.N = (int)a.N;
    t.H = a.H;
    t.by_bh = FastDiv((uint32_t)(a.B * a.H));
    t.by_h = FastDiv((uint32_t)a.H);
    t.by_g = FastDiv((uint32_t)a.G);
    t.W = a.W;
    t.S = a.S;
    t.SW = a.S > KB ? KB : (a.S + 15) / 16 * 16;
    t.half = a.r / 2;
    t.qtiles = (int)((a.N + 127) / 128);
    t.ntiles = t.qtiles * a.B * a.H;
    t.q = a.q;
    t.k = a.k;
    t.v = a.v;
    t.lse = a.lse;
    t.scale_log2 = a.scale_log2;
    t.status = a.status;
    cudaError_t e;
    t.split = t.half == 16;
    t.q_in = a.q;
    t.k_in = a.k;
    if (t.half) {
        const int64_t row = t.split ? 32 : D;
        t.q = Rows{scratch, a.H * a.N * row, a.N * row, row};
        t.k = Rows{static_cast<char*>(scratch) + win_fwd_q_bytes(a), a.Hkv * a.N * row, a.N * row, row};
        e = launch_win_rotate(a, t.q.p, t.k.p, t.split, s);
        if (e != cudaSuccess) return e;
    }
    CUtensorMap mq, mk, mv, msk, msv, mo, mqh, mkh, mskh;
    const uint32_t half_row = t.split ? 32 : 64;
    const uint64_t N = (uint64_t)a.N, B = (uint64_t)a.B, Hkv = (uint64_t)a.Hkv;
    const uint32_t sw = t.SW > 0 ? (uint32_t)t.SW : 16;
    bool ok = make_tmap_bf16_4d(&mq, t.q.p, N, (uint64_t)a.H, B, t.q.sn, t.q.sh, t.q.sb, 128, 4, half_row, half_row) &&
              make_tmap_bf16_4d(&mk, t.k.p, N, Hkv, B, t.k.sn, t.k.sh, t.k.sb, KB, 4, half_row, half_row) &&
              make_tmap_bf16_4d(&mv, t.v.p, N, Hkv, B, t.v.sn, t.v.sh, t.v.sb, KB) &&
              make_tmap_bf16_4d(&mo, a.out.p, N, (uint64_t)a.H, B, a.out.sn, a.out.sh, a.out.sb, 128);
    msk = mqh = mkh = mskh = mk;  // (where the kernel does not use them)
    msv = mv;
    if (ok && a.S > 0)
        ok = make_tmap_bf16_4d(&msk, t.k.p, N, Hkv, B, t.k.sn, t.k.sh, t.k.sb, sw, 4, half_row, half_row) &&
             // (ends with the sinks: the block's further rows are zeros, whatever those keys' values are)
             make_tmap_bf16_4d(&msv, t.v.p, (uint64_t)a.S, Hkv, B, t.v.sn, t.v.sh, t.v.sb, sw);
    if (ok && t.split)
        ok = make_tmap_bf16_4d(&mqh, a.q.p, N, (uint64_t)a.H, B, a.q.sn, a.q.sh, a.q.sb, 128, 4, 64, 32) &&
             make_tmap_bf16_4d(&mkh, a.k.p, N, Hkv, B, a.k.sn, a.k.sh, a.k.sb, KB, 4, 64, 32) &&
             (a.S == 0 || make_tmap_bf16_4d(&mskh, a.k.p, N, Hkv, B, a.k.sn, a.k.sh, a.k.sb, sw, 4, 64, 32));
    if (!ok) return cudaErrorInvalidValue;
    e = allow_smem<win_tc_kernel>(SMEM_BYTES);
    if (e != cudaSuccess) return e;
    const int nsm = sm_count(), grid = t.ntiles < nsm ? t.ntiles : nsm;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = t.half ? 1 : 0;  // (beside the rotation, which waited for all before it)
    return cudaLaunchKernelEx(&cfg, win_tc_kernel, mq, mk, mv, msk, msv, mo, mqh, mkh, mskh, t);
}

}  // namespace kvm
