// Sliding-window attention with sink tokens, backward, on the 5th-generation tensor
// cores (tcgen05 + TMEM + TMA).  bf16.
//
//   p_ij = 2^(s_ij log2 e - lse_i),  ds_ij = p_ij (dout_i . v_j - D_i),  D_i = dout_i . out_i
//   dq'_i = sum_j ds_ij k'_j / 8,  dk'_j = sum_i ds_ij q'_i / 8,  dv_j = sum_i p_ij dout_i
// with q', k' the rotated rows; dq and dk are rotated back as they leave.
//
// Two kernels, dq by query tiles and dk, dv by key tiles: seven products in the place
// of five, but every gradient row has one writer, so nothing is added through atomics
// and the same inputs give the same bits.  A pass before them rotates q and k into
// scratch; the first kernel leaves -lse and -D per query in blocks of 64 for the second.
//
// dq:     per 128 queries, key blocks of 64: S = Q K^T and dP = dO V^T (tensor memory), a
//         thread a query row makes dS in bf16 (tensor memory, two buffers), dQ += dS K
//         with dS read from tensor memory.  The next block's S and dP go out as soon as
//         this one's are in registers.
// dk, dv: per 128 keys, blocks of 64 queries of the G heads that share the key head, each
//         in two halves of 32, one a warpgroup's: S^T = K Q^T, dP^T = V dO^T, a thread a
//         key row; P^T and dS^T go over them as bf16 and are the tensor-memory operands of
//         dV += P^T dO and dK += dS^T Q: neither passes through shared memory.  One
//         half's products run while the other's rows work.
// Sinks: the queries behind the first key tile's window that still see keys j < S are
// cut into parts as long as a key tile's own work; each part writes its sums, a last
// kernel adds them to the tile's in a fixed order.
//
// 320 threads (producer, MMA issuer, two warpgroups of rows), 256 tensor-memory columns
// and under 113 KB of shared memory: two CTAs an SM, one's products beside the other's
// rows.  A block's chain of product, rows, product is what bounds it (tensor pipe 28%
// active, memory 24%), so the rows' part is kept short.  B4 H12 N8192 W512, the whole
// backward: 436 us (under a profiler: rotation pass 45, dq 160, dk and dv 234, sinks 6).  dk
// and dv with the products of a whole block at once take 13 us more, with one warpgroup of
// rows 31 more; without the wait of a half's products for the last readers of their place they
// took 10 less.
// All mbarrier waits are bounded; on expiry a CTA raises the status word, lets its copies
// and MMAs land, and exits.
#include <cuda.h>

#include "kvm_window.cuh"
#include "tc_primitives.cuh"

namespace kvm {
namespace winb {

using namespace tc;

constexpr int T = 128;            // rows of a tile
constexpr int BK = 64;            // rows of a block
constexpr int TILE = T * 128;     // bytes of [128][64] bf16
constexpr int BLK = BK * 128;
constexpr int NS = 3;             // stages
constexpr int NTHREADS = 320;
constexpr int NROWS = 256;        // threads of rows
constexpr int TMEM_COLS = 256;

struct BwdArgs {
    int N, H, Hkv, G, W, S, half;
    int tiles;                    // of 128 tokens
    int parts, part_blocks;       // sink parts of a key head, blocks of each
    int sink_q0;                  // first query of the sink parts, a multiple of 64
    FastDiv by_tiles, by_h, by_g; // tiles; query heads (dq) or key heads (dk, dv); G
    const float2* rope;
    Rows out, dout;
    const float* lse;
    float* nld;                   // per (b, h) and block of 64 queries: 64 of -lse, 64 of -D
    int nblk;                     // such blocks of a row
    float* part;                  // [B * Hkv][parts + 1][2][S][64]: dk', dv (fp32)
    float scale_log2, scale;
    int* status;
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ void drain(uint32_t bar, uint32_t parity) {
    const long long t0 = clock64();
    while (!mbar_try(bar, parity) && clock64() - t0 < (1ll << 28)) {
    }
}
__device__ __forceinline__ int clampi(int x, int hi) { return max(0, min(x, hi)); }
// bits [lo, hi) of 32
__device__ __forceinline__ uint32_t bits(int lo, int hi) {
    lo = clampi(lo, 32);
    hi = clampi(hi, 32);
    return (hi < 32 ? (1u << hi) - 1 : ~0u) & ~(lo < 32 ? (1u << lo) - 1 : ~0u);
}

// A row of 64 fp32 values times mul, rotated back at its position, as bf16 into a swizzled
// 128-byte row of shared memory.
__device__ __forceinline__ void put_row(float (&y)[64], float mul, const float2* cs_row, int half, uint8_t* row, int sw) {
#pragma unroll
    for (int x = 0; x < 64; ++x) y[x] *= mul;
    if (half == 16 || half == 32) {
#pragma unroll
        for (int x = 0; x < 16; ++x) {
            const float2 cs = cs_row[x];
            const int b = half == 16 ? x + 16 : x + 32;
            const float u = y[x], v = half == 16 ? y[x + 16] : y[x + 32];
            y[x] = u * cs.x + v * cs.y;
            if (b == x + 16)
                y[x + 16] = v * cs.x - u * cs.y;
            else
                y[x + 32] = v * cs.x - u * cs.y;
        }
        if (half == 32) {
#pragma unroll
            for (int x = 16; x < 32; ++x) {
                const float2 cs = cs_row[x];
                const float u = y[x], v = y[x + 32];
                y[x] = u * cs.x + v * cs.y;
                y[x + 32] = v * cs.x - u * cs.y;
            }
        }
    } else if (half > 0) {
        // (any other half: through local memory)
        float z[64];
#pragma unroll
        for (int x = 0; x < 64; ++x) z[x] = y[x];
#pragma unroll 1
        for (int x = 0; x < half; ++x) {
            const float2 cs = cs_row[x];
            const float u = z[x], v = z[x + half];
            z[x] = u * cs.x + v * cs.y;
            z[x + half] = v * cs.x - u * cs.y;
        }
#pragma unroll
        for (int x = 0; x < 64; ++x) y[x] = z[x];
    }
#pragma unroll
    for (int c = 0; c < 8; ++c)
        *reinterpret_cast<uint4*>(row + ((c ^ sw) << 4)) =
            make_uint4(pack2(y[8 * c], y[8 * c + 1]), pack2(y[8 * c + 2], y[8 * c + 3]), pack2(y[8 * c + 4], y[8 * c + 5]),
                       pack2(y[8 * c + 6], y[8 * c + 7]));
}
__device__ __forceinline__ void load_row(uint32_t taddr, float (&y)[64]) {
    uint32_t u[32], v[32];
    tmem_ld32(taddr, u);
    tmem_ld32(taddr + 32, v);
    tmem_wait_ld();
#pragma unroll
    for (int x = 0; x < 32; ++x) {
        y[x] = __uint_as_float(u[x]);
        y[32 + x] = __uint_as_float(v[x]);
    }
}

// ------------------------------------------------------------------------- dq
namespace q {
constexpr int OFF_Q = 0, OFF_DO = TILE, OFF_K = 2 * TILE, OFF_V = OFF_K + NS * BLK, OFF_D = OFF_V + NS * BLK, OFF_BAR = OFF_D + 2 * T * 4;
constexpr int SMEM = OFF_BAR + 256 + 1024;
constexpr int T_S = 0, T_DP = 64, T_DQ = 128, T_DS = 192;  // dS: two buffers of 32 columns
enum { B_Q = 0, B_FULL, B_EMPTY = B_FULL + NS, B_SPD = B_EMPTY + NS, B_FREE, B_DS, B_DONE, B_FINAL = B_DONE + 2, B_OUT, NBAR };

// the key blocks of a query tile: sinks, then from ws on
struct Keys {
    int ws, sink, n;
    __device__ __forceinline__ Keys(const BwdArgs& a, int q0) {
        const int q1 = min(q0 + T, a.N);
        ws = max(q0 - a.W + 1, 0);
        const bool own = a.S > 0 && q1 > a.W;  // the sinks are blocks of their own
        if (own) ws = max(ws, a.S);
        sink = own ? (a.S + BK - 1) / BK : 0;
        n = sink + (ws < q1 ? (q1 - ws + BK - 1) / BK : 0);
    }
    __device__ __forceinline__ int base(int j) const { return j < sink ? BK * j : ws + BK * (j - sink); }
};

__global__ void __launch_bounds__(NTHREADS, 2)
    win_dq_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                  const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const __grid_constant__ CUtensorMap tm_dq, const __grid_constant__ BwdArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto bar = [&](int i) { return smem_u32(bars + i); };
    const uint32_t sbase = smem_u32(sm);

    const int bh = a.by_tiles.div((int)blockIdx.x);
    const int q0 = (a.tiles - 1 - ((int)blockIdx.x - bh * a.tiles)) * T;
    const int b = a.by_h.div(bh), h = bh - b * a.H, hk = a.by_g.div(h);
    const Keys K(a, q0);

    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) mbar_init(bar(i), i == B_FREE || i == B_DS ? NROWS : i == B_OUT ? 128 : 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            mbar_expect_tx(bar(B_Q), 2 * TILE);
            tma_load_4d(sbase + OFF_Q, &tm_q, 0, q0, h, b, bar(B_Q));
            tma_load_4d(sbase + OFF_DO, &tm_do, 0, q0, h, b, bar(B_Q));
            int last = -1;
            for (int j = 0; j < K.n; ++j) {
                const int st = j % NS;
                if (j >= NS && !mbar_wait(bar(B_EMPTY + st), ((j / NS) - 1) & 1, abort_flag, a.status)) break;
                mbar_expect_tx(bar(B_FULL + st), 2 * BLK);
                tma_load_4d(sbase + OFF_K + st * BLK, &tm_k, 0, K.base(j), hk, b, bar(B_FULL + st));
                tma_load_4d(sbase + OFF_V + st * BLK, &tm_v, 0, K.base(j), hk, b, bar(B_FULL + st));
                last = j;
            }
            drain(bar(B_Q), 0);
            if (*abort_flag)
                for (int j = last; j >= 0 && j > last - NS; --j) drain(bar(B_FULL + j % NS), (j / NS) & 1);
        }
    } else if (warp == 1) {
        const bool lead = elect_one();
        const uint32_t id_s = idesc_bf16(T, BK, 0, 0), id_q = idesc_bf16(T, 64, 0, 1);
        const uint64_t dq = sdesc_sw128(sbase + OFF_Q, 16, 1024), ddo = sdesc_sw128(sbase + OFF_DO, 16, 1024);
        const uint64_t dk0 = sdesc_sw128(sbase + OFF_K, 16, 1024), dv0 = sdesc_sw128(sbase + OFF_V, 16, 1024);
        const uint64_t dm0 = sdesc_sw128(sbase + OFF_K, BLK, 1024);
        bool ok = mbar_wait_warp(bar(B_Q), 0, abort_flag, a.status);
        auto issue = [&](int j) -> bool {
            const int st = j % NS;
            if (!mbar_wait_warp(bar(B_FULL + st), (j / NS) & 1, abort_flag, a.status)) return false;
            tc_fence_after();
            const uint64_t dk = dk0 + st * (BLK >> 4), dv = dv0 + st * (BLK >> 4);
            if (lead) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16_ss(tmem + T_S, dq + 2 * ks, dk + 2 * ks, id_s, ks > 0);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16_ss(tmem + T_DP, ddo + 2 * ks, dv + 2 * ks, id_s, ks > 0);
                mma_commit(bar(B_SPD));
            }
            __syncwarp();
            return true;
        };
        if (ok) ok = issue(0);
        for (int j = 0; ok && j < K.n; ++j) {
            const int st = j % NS;
            // S and dP of block j are in registers: the next block's may take their place
            if (!mbar_wait_warp(bar(B_FREE), j & 1, abort_flag, a.status)) break;
            if (j + 1 < K.n && !issue(j + 1)) break;
            if (!mbar_wait_warp(bar(B_DS), j & 1, abort_flag, a.status)) break;
            tc_fence_after();
            const uint64_t dm = dm0 + st * (BLK >> 4);
            const uint32_t ds = tmem + T_DS + 32 * (j & 1);
            if (lead) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) mma_bf16_ts(tmem + T_DQ, ds + 8 * ks, dm + 128 * ks, id_q, (j > 0 || ks > 0) ? 1u : 0u);
                mma_commit(bar(B_DONE + (j & 1)));
                mma_commit(bar(B_EMPTY + st));
            }
            __syncwarp();
        }
        if (lead) mma_commit(bar(B_FINAL));  // every MMA completes before the tensor memory is released
        drain(bar(B_FINAL), 0);
    } else {
        const int wg = (warp - 2) >> 2, c0 = 32 * wg;   // keys [c0, c0 + 32) of each block
        const int wq = warp & 3, row = wq * 32 + lane;  // query row = tensor-memory lane
        const uint32_t lb = tmem + ((uint32_t)(wq * 32) << 16);
        const int p = q0 + row;
        // D: each warpgroup half of the row
        float part_d = 0.f, nl = -INFINITY;  // (a query past the last one has probability 0)
        if (p < a.N) {
            nl = -a.lse[(int64_t)bh * a.N + p];
            const uint4* o4 = reinterpret_cast<const uint4*>(a.out.at<const __nv_bfloat16>(b, h, p)) + 4 * wg;
            const uint4* g4 = reinterpret_cast<const uint4*>(a.dout.at<const __nv_bfloat16>(b, h, p)) + 4 * wg;
            uint4 o[4], g[4];
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                o[x] = o4[x];
                g[x] = g4[x];
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                const uint32_t ow[4] = {o[x].x, o[x].y, o[x].z, o[x].w}, gw[4] = {g[x].x, g[x].y, g[x].z, g[x].w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    part_d = fmaf(__uint_as_float(ow[u] << 16), __uint_as_float(gw[u] << 16), part_d);
                    part_d = fmaf(__uint_as_float(ow[u] & 0xffff0000u), __uint_as_float(gw[u] & 0xffff0000u), part_d);
                }
            }
        }
        float* const halves = reinterpret_cast<float*>(sm + OFF_D);
        halves[wg * T + row] = part_d;
        asm volatile("bar.sync 1, 256;" ::: "memory");  // (every thread of rows comes here, before any wait)
        const float nd = -(halves[row] + halves[T + row]);
        if (wg == 0 && (p >> 6) < a.nblk) {
            float* nld = a.nld + ((int64_t)bh * a.nblk + (p >> 6)) * 128 + (p & 63);
            nld[0] = nl;
            nld[64] = nd;
        }
        const float2 sl2 = make_float2(a.scale_log2, a.scale_log2), nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
        bool ok = true;
        for (int j = 0; j < K.n; ++j) {
            const bool sink = j < K.sink;
            const int key0 = K.base(j), w0 = q0 + wq * 32 - key0 + 1;
            const int top = sink ? min(BK, a.S - key0) : BK, off = sink ? 1 << 30 : a.W;
            // columns [lo, hi) are keys that this query sees
            const int hi = min(w0 + lane, top), lo = w0 + lane - off;
            if (!mbar_wait_warp(bar(B_SPD), j & 1, abort_flag, a.status)) { ok = false; break; }
            tc_fence_after();
            uint32_t dw[2][8];
            if (c0 >= min(w0 + 31, top) || c0 + 32 <= w0 - off) {  // none of the warp's rows sees these keys
#pragma unroll
                for (int x = 0; x < 8; ++x) dw[0][x] = dw[1][x] = 0;
            } else {
                const bool part = c0 + 32 > min(w0, top) || c0 < w0 + 31 - off;
                const uint32_t seen = bits(lo - c0, hi - c0);
#pragma unroll
                for (int x2 = 0; x2 < 2; ++x2) {
                    uint32_t s[16], d[16];
                    tmem_ld16(lb + T_S + c0 + 16 * x2, s);
                    tmem_ld16(lb + T_DP + c0 + 16 * x2, d);
                    tmem_wait_ld();
                    if (part) {
#pragma unroll
                        for (int x = 0; x < 16; ++x)
                            if (!(seen & (1u << (16 * x2 + x)))) s[x] = __float_as_uint(-INFINITY);
                    }
#pragma unroll
                    for (int x = 0; x < 16; x += 2) {
                        const float2 t = __ffma2_rn(make_float2(__uint_as_float(s[x]), __uint_as_float(s[x + 1])), sl2, nl2);
                        const float2 e = make_float2(ex2(t.x), ex2(t.y));
                        const float2 g = __fmul2_rn(e, __fadd2_rn(make_float2(__uint_as_float(d[x]), __uint_as_float(d[x + 1])), nd2));
                        dw[x2][x >> 1] = pack2(g.x, g.y);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(bar(B_FREE));
            // the buffer's last reader, dQ of block j - 2, is done
            if (j >= 2 && !mbar_wait_warp(bar(B_DONE + (j & 1)), ((j >> 1) - 1) & 1, abort_flag, a.status)) { ok = false; break; }
            tc_fence_after();
            tmem_st8(lb + T_DS + 32 * (j & 1) + 16 * wg, dw[0]);
            tmem_st8(lb + T_DS + 32 * (j & 1) + 16 * wg + 8, dw[1]);
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(B_DS));
        }
        if (ok) ok = mbar_wait_warp(bar(B_DONE + ((K.n - 1) & 1)), ((K.n - 1) >> 1) & 1, abort_flag, a.status);
        if (ok && wg == 0) {
            tc_fence_after();
            float y[64];
            load_row(lb + T_DQ, y);
            put_row(y, a.scale, a.rope + (int64_t)min(p, a.N - 1) * a.half, a.half, sm + OFF_Q + row * 128, row & 7);
            fence_proxy_async();
            mbar_arrive(bar(B_OUT));
            if (warp == 2 && lane == 0 && mbar_wait(bar(B_OUT), 0, abort_flag, a.status)) {
                tma_store_4d(&tm_dq, sbase + OFF_Q, 0, q0, h, b);
                bulk_commit();
                bulk_wait_all();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}
}  // namespace q

// --------------------------------------------------------------------- dk, dv
namespace kv {
constexpr int OFF_K = 0, OFF_V = TILE, OFF_Q = 2 * TILE, OFF_DO = OFF_Q + NS * BLK, OFF_LD = OFF_DO + NS * BLK;
constexpr int OFF_BAR = OFF_LD + NS * 512, SMEM = OFF_BAR + 256 + 1024;
constexpr int T_S = 0, T_DP = 64, T_DV = 128, T_DK = 192;  // P^T over S^T, dS^T over dP^T
enum { B_KV = 0, B_FULL, B_EMPTY = B_FULL + NS, B_SPD = B_EMPTY + NS, B_P = B_SPD + 2, B_READ = B_P + 2, B_DONE = B_READ + 2, B_OUT, NBAR };

__global__ void __launch_bounds__(NTHREADS, 2)
    win_dkv_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                   const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                   const __grid_constant__ CUtensorMap tm_dk, const __grid_constant__ CUtensorMap tm_dv,
                   const __grid_constant__ BwdArgs a) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + OFF_BAR);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBAR);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto bar = [&](int i) { return smem_u32(bars + i); };
    const uint32_t sbase = smem_u32(sm);

    // a key head's items: its key tiles, then its sink parts
    const int bk = a.by_tiles.div((int)blockIdx.x), item = (int)blockIdx.x - bk * (a.tiles + a.parts);
    const int b = a.by_h.div(bk), hk = bk - b * a.Hkv;
    const bool sink = item >= a.tiles;
    const int k0 = sink ? 0 : item * T;
    // blocks of 64 queries from qb on, nq of them per head, [i0, i1) of the G heads' list
    const int qb = sink ? a.sink_q0 / BK : k0 / BK;
    const int nq = (sink ? (a.N + BK - 1) / BK : (min(a.N, k0 + T - 1 + a.W) + BK - 1) / BK) - qb;
    const int i0 = sink ? (item - a.tiles) * a.part_blocks : 0, i1 = sink ? min(i0 + a.part_blocks, nq * a.G) : nq * a.G;
    const int n = i1 - i0;  // >= 1
    int g0 = sink ? i0 / nq : 0, x0 = i0 - g0 * nq;  // first block's head and place
    auto next = [&](int& g, int& x) {
        if (++x == nq) x = 0, ++g;
    };

    if (tid == 0) {
        for (int i = 0; i < NBAR; ++i) mbar_init(bar(i), i == B_P || i == B_P + 1 ? 128 : i == B_OUT ? NROWS : 1);
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 1) tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            mbar_expect_tx(bar(B_KV), 2 * TILE);
            tma_load_4d(sbase + OFF_K, &tm_k, 0, k0, hk, b, bar(B_KV));
            tma_load_4d(sbase + OFF_V, &tm_v, 0, k0, hk, b, bar(B_KV));
            int last = -1, g = g0, x = x0;
            for (int j = 0; j < n; ++j) {
                const int st = j % NS;
                if (j >= NS && !mbar_wait(bar(B_EMPTY + st), ((j / NS) - 1) & 1, abort_flag, a.status)) break;
                const int h = hk * a.G + g;
                mbar_expect_tx(bar(B_FULL + st), 2 * BLK + 512);
                tma_load_4d(sbase + OFF_Q + st * BLK, &tm_q, 0, (qb + x) * BK, h, b, bar(B_FULL + st));
                tma_load_4d(sbase + OFF_DO + st * BLK, &tm_do, 0, (qb + x) * BK, h, b, bar(B_FULL + st));
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], 512, [%2];" ::"r"(
                                 sbase + OFF_LD + st * 512),
                             "l"(a.nld + (((int64_t)b * a.H + h) * a.nblk + qb + x) * 128), "r"(bar(B_FULL + st))
                             : "memory");
                last = j;
                next(g, x);
            }
            drain(bar(B_KV), 0);
            if (*abort_flag)
                for (int j = last; j >= 0 && j > last - NS; --j) drain(bar(B_FULL + j % NS), (j / NS) & 1);
        }
    } else if (warp == 1) {
        const bool lead = elect_one();
        const uint32_t id_s = idesc_bf16(T, 32, 0, 0), id_o = idesc_bf16(T, 64, 0, 1);
        const uint64_t dk = sdesc_sw128(sbase + OFF_K, 16, 1024), dv = sdesc_sw128(sbase + OFF_V, 16, 1024);
        const uint64_t dq0 = sdesc_sw128(sbase + OFF_Q, 16, 1024), ddo0 = sdesc_sw128(sbase + OFF_DO, 16, 1024);
        const uint64_t mq0 = sdesc_sw128(sbase + OFF_Q, BLK, 1024), mdo0 = sdesc_sw128(sbase + OFF_DO, BLK, 1024);
        bool ok = mbar_wait_warp(bar(B_KV), 0, abort_flag, a.status);
        // by halves of 32 queries, the warpgroups' in turn: half s's S^T and dP^T go out once half
        // s - 2's products have read P^T and dS^T there (the tensor core keeps the order of
        // products only where they share shape and accumulator), then half s - 1's dV and dK once
        // its rows are done
        for (int s = 0; ok && s <= 2 * n; ++s) {
            if (s < 2 * n) {
                const int j = s >> 1, st = j % NS, hf = s & 1;
                if (!hf && !mbar_wait_warp(bar(B_FULL + st), (j / NS) & 1, abort_flag, a.status)) break;
                if (j > 0 && !mbar_wait_warp(bar(B_READ + hf), (j - 1) & 1, abort_flag, a.status)) break;
                tc_fence_after();
                const uint64_t off = st * (BLK >> 4) + hf * (32 * 128 >> 4);
                const uint32_t tS = tmem + T_S + 32 * hf, tD = tmem + T_DP + 32 * hf;
                if (lead) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) mma_bf16_ss(tS, dk + 2 * ks, dq0 + off + 2 * ks, id_s, ks > 0);
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) mma_bf16_ss(tD, dv + 2 * ks, ddo0 + off + 2 * ks, id_s, ks > 0);
                    mma_commit(bar(B_SPD + hf));
                }
                __syncwarp();
            }
            if (s > 0) {
                const int j = (s - 1) >> 1, st = j % NS, hf = (s - 1) & 1;
                if (!mbar_wait_warp(bar(B_P + hf), j & 1, abort_flag, a.status)) break;
                tc_fence_after();
                const uint64_t off = st * (BLK >> 4) + hf * 256;
                const uint32_t tS = tmem + T_S + 32 * hf, tD = tmem + T_DP + 32 * hf;
                if (lead) {
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) mma_bf16_ts(tmem + T_DV, tS + 8 * ks, mdo0 + off + 128 * ks, id_o, (s > 1 || ks > 0) ? 1u : 0u);
#pragma unroll
                    for (int ks = 0; ks < 2; ++ks) mma_bf16_ts(tmem + T_DK, tD + 8 * ks, mq0 + off + 128 * ks, id_o, (s > 1 || ks > 0) ? 1u : 0u);
                    mma_commit(bar(B_READ + hf));
                    if (hf) mma_commit(bar(B_EMPTY + st));
                }
                __syncwarp();
            }
        }
        if (lead) mma_commit(bar(B_DONE));  // every MMA completes before the tensor memory is read out or released
        drain(bar(B_DONE), 0);
    } else {
        const int wg = (warp - 2) >> 2, c0 = 32 * wg;   // queries [c0, c0 + 32) of each block
        const int wq = warp & 3, row = wq * 32 + lane;  // key row = tensor-memory lane
        const uint32_t lb = tmem + ((uint32_t)(wq * 32) << 16);
        const int kb = k0 + wq * 32, key = kb + lane;
        const float2 sl2 = make_float2(a.scale_log2, a.scale_log2);
        const bool idle = sink && kb >= a.S;  // (none of the warp's keys is a sink)
        bool ok = true;
        int g = g0, x = x0;
        for (int j = 0; j < n; ++j) {
            const int st = j % NS, q0 = (qb + x) * BK;
            next(g, x);
            if (!mbar_wait_warp(bar(B_SPD + wg), j & 1, abort_flag, a.status)) { ok = false; break; }
            tc_fence_after();
            // queries that see the warp's keys: window i in [key, key + W), sinks i >= key + W
            const int lo = sink ? (key < a.S ? key + a.W - q0 : BK) : key - q0, hi = sink ? BK : key + a.W - q0;
            const int lo0 = sink ? kb + a.W - q0 : kb - q0, lo1 = sink && kb + 31 >= a.S ? BK : lo0 + 31;
            const int hi0 = sink ? BK : kb + a.W - q0, hi1 = sink ? BK : hi0 + 31;
            const float* ld = reinterpret_cast<const float*>(sm + OFF_LD + st * 512);
            const bool dead = idle || c0 + 32 <= lo0 || c0 >= hi1, part = c0 < lo1 || c0 + 32 > hi0;
            const uint32_t seen = bits(lo - c0, hi - c0);
#pragma unroll
            for (int x2 = 0; x2 < 2; ++x2) {
                const int c = c0 + 16 * x2;
                uint32_t pw[8], dw[8];
                if (dead) {
#pragma unroll
                    for (int u = 0; u < 8; ++u) pw[u] = dw[u] = 0;
                } else {
                    uint32_t s[16], d[16];
                    tmem_ld16(lb + T_S + c, s);
                    tmem_ld16(lb + T_DP + c, d);
                    tmem_wait_ld();
                    if (part) {
#pragma unroll
                        for (int u = 0; u < 16; ++u)
                            if (!(seen & (1u << (16 * x2 + u)))) s[u] = __float_as_uint(-INFINITY);
                    }
#pragma unroll
                    for (int u = 0; u < 16; u += 4) {
                        const float4 l4 = *reinterpret_cast<const float4*>(ld + c + u);
                        const float4 d4 = *reinterpret_cast<const float4*>(ld + 64 + c + u);
#pragma unroll
                        for (int v = 0; v < 4; v += 2) {
                            const float2 nl = v ? make_float2(l4.z, l4.w) : make_float2(l4.x, l4.y);
                            const float2 nd = v ? make_float2(d4.z, d4.w) : make_float2(d4.x, d4.y);
                            const float2 t = __ffma2_rn(make_float2(__uint_as_float(s[u + v]), __uint_as_float(s[u + v + 1])), sl2, nl);
                            const float2 e = make_float2(ex2(t.x), ex2(t.y));
                            const float2 f = __fmul2_rn(e, __fadd2_rn(make_float2(__uint_as_float(d[u + v]), __uint_as_float(d[u + v + 1])), nd));
                            pw[(u + v) >> 1] = pack2(e.x, e.y);
                            dw[(u + v) >> 1] = pack2(f.x, f.y);
                        }
                    }
                }
                // over this warpgroup's own columns of S^T and dP^T, behind what is still to be read
                tmem_st8(lb + T_S + c0 + 8 * x2, pw);
                tmem_st8(lb + T_DP + c0 + 8 * x2, dw);
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(B_P + wg));
        }
        if (ok) ok = mbar_wait_warp(bar(B_DONE), 0, abort_flag, a.status);
        if (ok) {
            tc_fence_after();
            // the first warpgroup takes dv, the second dk (the K and V tiles are read no more)
            float y[64];
            const bool parted = a.parts > 0 && k0 == 0 && kb < a.S;  // sums of the sinks go to a part
            float* part = a.part + ((((int64_t)bk * (a.parts + 1) + (sink ? item - a.tiles + 1 : 0)) * 2 + (1 - wg)) * a.S + key) * D;
            load_row(lb + (wg ? T_DK : T_DV), y);
            if (parted && key < a.S) {
#pragma unroll
                for (int u = 0; u < 64; u += 4) *reinterpret_cast<float4*>(part + u) = make_float4(y[u], y[u + 1], y[u + 2], y[u + 3]);
            }
            __syncwarp();
            if (!sink) {
                if (wg == 0)
                    put_row(y, 1.f, nullptr, 0, sm + OFF_V + row * 128, row & 7);
                else
                    put_row(y, a.scale, a.rope + (int64_t)min(key, a.N - 1) * a.half, a.half, sm + OFF_K + row * 128, row & 7);
                fence_proxy_async();
                mbar_arrive(bar(B_OUT));
                if (warp == 2 && lane == 0 && mbar_wait(bar(B_OUT), 0, abort_flag, a.status)) {
                    tma_store_4d(&tm_dk, sbase + OFF_K, 0, k0, hk, b);
                    tma_store_4d(&tm_dv, sbase + OFF_V, 0, k0, hk, b);
                    bulk_commit();
                    bulk_wait_all();
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}
}  // namespace kv

// The sinks' rows from the parts, a CTA a row: a warp takes every JW-th part, two dims a lane,
// and the warps are added up in their order (one warp a row: 10 us more for the backward of B1
// H16/4 N30011 W1024, 691 us).
constexpr int JW = 8;
template <typename E>
__global__ void __launch_bounds__(32 * JW) win_sink_kernel(Rows dk, Rows dv, const float* part, int parts, int S, int Hkv, int half,
                                                       const float2* rope, float scale) {
    __shared__ float sums[JW][4][32];
    const int w = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int j = w % S, bk = w / S;
    const float* p = part + (((int64_t)bk * (parts + 1) + warp) * 2 * S + j) * D;
    float k[2] = {0.f, 0.f}, v[2] = {0.f, 0.f};
#pragma unroll 8
    for (int x = warp; x <= parts; x += JW, p += 2 * JW * (int64_t)S * D) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            k[u] += p[lane + 32 * u];
            v[u] += p[(int64_t)S * D + lane + 32 * u];
        }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        sums[warp][u][lane] = k[u];
        sums[warp][2 + u][lane] = v[u];
    }
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int x = 1; x < JW; ++x)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            k[u] += sums[x][u][lane];
            v[u] += sums[x][2 + u][lane];
        }
    float y[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int d = lane + 32 * u, pd = d < half ? d + half : d - half;
        const float e0 = __shfl_sync(0xffffffffu, k[0], pd & 31), e1 = __shfl_sync(0xffffffffu, k[1], pd & 31);
        y[u] = k[u] * scale;
        if (d < 2 * half) {
            const float2 cs = rope[j * half + (d < half ? d : pd)];
            const float me = k[u] * scale, other = (pd < 32 ? e0 : e1) * scale;
            y[u] = d < half ? me * cs.x + other * cs.y : me * cs.x - other * cs.y;
        }
    }
    E *ok = dk.at<E>(bk / Hkv, bk % Hkv, j), *ov = dv.at<E>(bk / Hkv, bk % Hkv, j);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        ok[lane + 32 * u] = from_f<E>(y[u]);
        ov[lane + 32 * u] = from_f<E>(v[u]);
    }
}

}  // namespace winb

// scratch of the tensor-core backward: offsets, and the sink parts
WinBwdPlan win_bwd_plan(const WinArgs& a) {
    WinBwdPlan p{};
    const int64_t N = a.N;
    p.nblk = (int)((N + 63) / 64);
    if (a.S > 0 && N > a.W) {
        const int64_t q0 = a.W / 64 * 64, blocks = ((N + 63) / 64 - q0 / 64) * a.G;
        int64_t per = (int64_t)a.G * ((a.W + 127) / 64 + 1);  // a key tile's own
        if (blocks > per * 256) per = (blocks + 255) / 256;
        p.part_blocks = (int)per;
        p.parts = (int)((blocks + per - 1) / per);
        p.sink_q0 = (int)q0;
    }
    size_t o = 0;
    auto take = [&](size_t bytes) { size_t at = o; o = (o + bytes + 255) / 256 * 256; return at; };
    const size_t rq = (size_t)a.B * a.H * N * D * 2, rk = (size_t)a.B * a.Hkv * N * D * 2;
    p.q_rot = take(a.r ? rq : 0);
    p.k_rot = take(a.r ? rk : 0);
    p.nld = take((size_t)a.B * a.H * p.nblk * 512);
    p.part = take(p.parts ? (size_t)a.B * a.Hkv * (p.parts + 1) * 2 * a.S * D * 4 : 0);
    p.total = o;
    return p;
}

cudaError_t launch_win_bwd_tc(const WinArgs& a, void* scratch, cudaStream_t s) {
    using namespace winb;
    const WinBwdPlan pl = win_bwd_plan(a);
    char* sc = static_cast<char*>(scratch);
    Rows q = a.q, k = a.k;
    cudaError_t e = cudaSuccess;
    if (a.r) {
        q = Rows{sc + pl.q_rot, (int64_t)a.H * a.N * D, a.N * D, D};
        k = Rows{sc + pl.k_rot, (int64_t)a.Hkv * a.N * D, a.N * D, D};
        e = launch_win_rotate(a, q.p, k.p, false, s);
        if (e != cudaSuccess) return e;
    }
    float* nld = reinterpret_cast<float*>(sc + pl.nld);
    BwdArgs t{};
    t.N = (int)a.N;
    t.H = a.H;
    t.Hkv = a.Hkv;
    t.G = a.G;
    t.W = a.W;
    t.S = a.S;
    t.half = a.r / 2;
    t.tiles = (int)((a.N + T - 1) / T);
    t.by_tiles = FastDiv((uint32_t)t.tiles);
    t.by_h = FastDiv((uint32_t)a.H);
    t.by_g = FastDiv((uint32_t)a.G);
    t.rope = a.rope;
    t.out = a.out;
    t.dout = a.dout;
    t.lse = a.lse;
    t.nld = nld;
    t.nblk = pl.nblk;
    t.scale_log2 = a.scale_log2;
    t.scale = a.scale;
    t.status = a.status;
    const uint64_t N = (uint64_t)a.N, B = (uint64_t)a.B, H = (uint64_t)a.H, Hkv = (uint64_t)a.Hkv;
    CUtensorMap mq, mdo, mk, mv, mo, mo2;
    if (!make_tmap_bf16_4d(&mq, q.p, N, H, B, q.sn, q.sh, q.sb, T) ||
        !make_tmap_bf16_4d(&mdo, a.dout.p, N, H, B, a.dout.sn, a.dout.sh, a.dout.sb, T) ||
        !make_tmap_bf16_4d(&mk, k.p, N, Hkv, B, k.sn, k.sh, k.sb, BK) ||
        !make_tmap_bf16_4d(&mv, a.v.p, N, Hkv, B, a.v.sn, a.v.sh, a.v.sb, BK) ||
        !make_tmap_bf16_4d(&mo, a.dq.p, N, H, B, a.dq.sn, a.dq.sh, a.dq.sb, T))
        return cudaErrorInvalidValue;
    e = allow_smem<q::win_dq_kernel>(q::SMEM);
    if (e == cudaSuccess) e = allow_smem<kv::win_dkv_kernel>(kv::SMEM);
    if (e != cudaSuccess) return e;
    q::win_dq_kernel<<<(unsigned)(t.tiles * a.B * a.H), NTHREADS, q::SMEM, s>>>(mq, mdo, mk, mv, mo, t);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;

    t.parts = pl.parts;
    t.part_blocks = pl.part_blocks;
    t.sink_q0 = pl.sink_q0;
    t.part = reinterpret_cast<float*>(sc + pl.part);
    t.by_tiles = FastDiv((uint32_t)(t.tiles + t.parts));
    t.by_h = FastDiv((uint32_t)a.Hkv);
    if (!make_tmap_bf16_4d(&mq, q.p, N, H, B, q.sn, q.sh, q.sb, BK) ||
        !make_tmap_bf16_4d(&mdo, a.dout.p, N, H, B, a.dout.sn, a.dout.sh, a.dout.sb, BK) ||
        !make_tmap_bf16_4d(&mk, k.p, N, Hkv, B, k.sn, k.sh, k.sb, T) ||
        !make_tmap_bf16_4d(&mv, a.v.p, N, Hkv, B, a.v.sn, a.v.sh, a.v.sb, T) ||
        !make_tmap_bf16_4d(&mo, a.dk.p, N, Hkv, B, a.dk.sn, a.dk.sh, a.dk.sb, T) ||
        !make_tmap_bf16_4d(&mo2, a.dv.p, N, Hkv, B, a.dv.sn, a.dv.sh, a.dv.sb, T))
        return cudaErrorInvalidValue;
    kv::win_dkv_kernel<<<(unsigned)((t.tiles + t.parts) * a.B * a.Hkv), NTHREADS, kv::SMEM, s>>>(mq, mdo, mk, mv, mo, mo2, t);
    e = cudaGetLastError();
    if (e != cudaSuccess || !t.parts) return e;
    return launch_win_sinks(a, t.part, t.parts, true, s);
}

cudaError_t launch_win_sinks(const WinArgs& a, const float* part, int parts, bool bf16, cudaStream_t s) {
    const unsigned grid = (unsigned)(a.B * a.Hkv * a.S);
    if (bf16)
        winb::win_sink_kernel<__nv_bfloat16><<<grid, 32 * winb::JW, 0, s>>>(a.dk, a.dv, part, parts, a.S, a.Hkv, a.r / 2, a.rope, a.scale);
    else
        winb::win_sink_kernel<float><<<grid, 32 * winb::JW, 0, s>>>(a.dk, a.dv, part, parts, a.S, a.Hkv, a.r / 2, a.rope, a.scale);
    return cudaGetLastError();
}

}  // namespace kvm
