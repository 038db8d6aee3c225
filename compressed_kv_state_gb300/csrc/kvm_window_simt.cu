// Sliding-window attention with sink tokens in fp32 arithmetic: the forward, and
// the backward in two kernels (dq by query tiles, dk and dv by key tiles).
//
//   s_ij = q'_i . k'_j / 8 for j <= i and (i - j < W or j < S), p = softmax_j(s),
//   out_i = sum_j p_ij v_j;   D_i = dout_i . out_i,
//   ds_ij = p_ij (dout_i . v_j - D_i) / 8,  dq'_i = sum_j ds_ij k'_j,
//   dk'_j = sum_i ds_ij q'_i,  dv_j = sum_i p_ij dout_i
// with q', k' the rotated rows; dq, dk are rotated back.
//
// Tiles of 64 queries x 64 keys in shared memory, 256 threads of 4 x 4 (or 4 x 4
// dims) each: every product is 64 x 64 x 64 with two 16-byte shared loads per
// 16 multiply-adds of a thread (two at once).  The next tiles come in by asynchronous
// copies beside a tile's products.  Two CTAs an SM, so 128 registers (with the 148 that the
// compiler takes otherwise one fits: 1,530 us for the backward below), at which each kernel
// spills a little (28, 24 and 52 bytes stored).  B2 H8/2 N4096 W512 S16 r32: forward 338 us
// (24.5 TFLOP/s; 372 without the copies ahead), backward 1,092 (18.9).  No unit is near its
// limit (the multiply-add pipe is 40% busy): what is left are the latencies of shared loads and
// barriers.  Sums are made in a fixed order.  fp32 layers run here: the tensor cores' own
// fp32 form keeps 10 bits of an operand.
#include "kvm_window.cuh"

namespace kvm {
namespace wins {

constexpr int T64 = 64;
constexpr int LD = 68;  // row stride in floats: 16 rows read by a quarter warp fall in distinct banks
constexpr int TILE_F = T64 * LD;
constexpr int NT = 256;

// rows [n0, n0 + 64) of one (b, h) into a tile (fp32), rows at or past n1 zero
__device__ __forceinline__ void load_tile(float* dst, const float* base, int64_t sn, int64_t n0, int64_t n1) {
    for (int i = threadIdx.x; i < T64 * 16; i += NT) {
        const int row = i >> 4, c = (i & 15) * 4;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (n0 + row < n1) x = *reinterpret_cast<const float4*>(base + (n0 + row) * sn + c);
        *reinterpret_cast<float4*>(dst + row * LD + c) = x;
    }
}
// The same without waiting (16-byte copies, zeros where n1 ends): landed() and a barrier before it is read.
__device__ __forceinline__ void fetch_tile(float* dst, const float* base, int64_t sn, int64_t n0, int64_t n1) {
    for (int i = threadIdx.x; i < T64 * 16; i += NT) {
        const int row = i >> 4, c = (i & 15) * 4;
        const bool in = n0 + row < n1;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(dst + row * LD + c)),
                     "l"(in ? base + (n0 + row) * sn + c : base), "r"(in ? 16 : 0)
                     : "memory");
    }
}
__device__ __forceinline__ void landed() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// rotate-half of a tile's rows at positions n0 + row (sign -1: back)
__device__ __forceinline__ void rotate_tile(float* t, int64_t n0, int64_t n1, const float2* rope, int half,
                                            float sign) {
    const int row = threadIdx.x >> 2;  // four threads a row
    if (n0 + row >= n1) return;
    for (int x = threadIdx.x & 3; x < half; x += 4) {
        const float2 cs = rope[(n0 + row) * half + x];
        const float s = sign * cs.y;
        float* p = t + row * LD + x;
        const float a = p[0], b = p[half];
        p[0] = a * cs.x - b * s;
        p[half] = b * cs.x + a * s;
    }
}

// c[i][j] = A[ty + 16 i] . B[tx + 16 j]
__device__ __forceinline__ void mm_nt(float (&c)[4][4], const float* A, const float* B, int ty, int tx) {
    float2 s[4][4];  // the sums over even and odd k
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < D; k += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) a[i] = *reinterpret_cast<const float4*>(A + (ty + 16 * i) * LD + k);
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = *reinterpret_cast<const float4*>(B + (tx + 16 * j) * LD + k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = __ffma2_rn(make_float2(a[i].x, a[i].y), make_float2(b[j].x, b[j].y), s[i][j]);
                s[i][j] = __ffma2_rn(make_float2(a[i].z, a[i].w), make_float2(b[j].z, b[j].w), s[i][j]);
            }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[i][j] = s[i][j].x + s[i][j].y;
}
// a += p * v
__device__ __forceinline__ void add2(float (&a)[4], float p, const float4& v) {
    const float2 lo = __ffma2_rn(make_float2(p, p), make_float2(v.x, v.y), make_float2(a[0], a[1]));
    const float2 hi = __ffma2_rn(make_float2(p, p), make_float2(v.z, v.w), make_float2(a[2], a[3]));
    a[0] = lo.x, a[1] = lo.y, a[2] = hi.x, a[3] = hi.y;
}
// acc[i][0..3] += sum_k P[ty + 16 i][k] * V[k][4 tx ..]; skip: a weight of -0 hides its row of V
// (a masked key's value may be anything; a key that is seen has a weight of +0 at least, and one
// too small for fp32 does not hide that its value is not finite)
template <bool SKIP>
__device__ __forceinline__ void mm_nn(float (&acc)[4][4], const float* P, const float* V, int ty, int tx) {
#pragma unroll 2
    for (int k = 0; k < T64; k += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = *reinterpret_cast<const float4*>(P + (ty + 16 * i) * LD + k);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const float4 v = *reinterpret_cast<const float4*>(V + (k + x) * LD + 4 * tx);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float w = x == 0 ? p[i].x : x == 1 ? p[i].y : x == 2 ? p[i].z : p[i].w;
                if (SKIP && __float_as_uint(w) == 0x80000000u) continue;
                add2(acc[i], w, v);
            }
        }
    }
}
// acc[i][0..3] += sum_q P[q][4 ty + i] * X[q][4 tx ..]
__device__ __forceinline__ void mm_tn(float (&acc)[4][4], const float* P, const float* X, int ty, int tx) {
#pragma unroll 4
    for (int q = 0; q < T64; ++q) {
        const float4 p = *reinterpret_cast<const float4*>(P + q * LD + 4 * ty);
        const float4 x = *reinterpret_cast<const float4*>(X + q * LD + 4 * tx);
        const float pw[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            add2(acc[i], pw[i], x);
        }
    }
}
// 4 x 4 values into rows row(i), dims 4 tx .. of a tile
template <class F> __device__ __forceinline__ void put_tile(float* t, const float (&v)[4][4], F row, int tx) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<float4*>(t + row(i) * LD + 4 * tx) = make_float4(v[i][0], v[i][1], v[i][2], v[i][3]);
}
__device__ __forceinline__ void store_tile(const float* t, float* base, int64_t sn, int64_t n0, int64_t n1, float mul) {
    for (int i = threadIdx.x; i < T64 * 16; i += NT) {
        const int row = i >> 4, c = (i & 15) * 4;
        if (n0 + row >= n1) continue;
        const float4 s = *reinterpret_cast<const float4*>(t + row * LD + c);
        *reinterpret_cast<float4*>(base + (n0 + row) * sn + c) = make_float4(s.x * mul, s.y * mul, s.z * mul, s.w * mul);
    }
}

__device__ __forceinline__ bool visible(int64_t i, int64_t j, int W, int S) { return j <= i && (i - j < W || j < S); }

// the key tiles a 64-query tile sees: sinks before its window, then the window
struct KeyTiles {
    int64_t ws, q_end;
    int nsink, n;
    __device__ KeyTiles(int64_t q0, int64_t N, int W, int S) {
        ws = q0 - W + 1 > 0 ? q0 - W + 1 : 0;
        q_end = q0 + T64 < N ? q0 + T64 : N;
        const int64_t sinks = S < ws ? S : ws;
        nsink = (int)((sinks + T64 - 1) / T64);
        n = nsink + (int)((q_end - ws + T64 - 1) / T64);
    }
    // tile t covers keys [k0, k1)
    __device__ void at(int t, int S, int64_t& k0, int64_t& k1) const {
        if (t < nsink) {
            k0 = (int64_t)t * T64;
            k1 = S < ws ? S : ws;
        } else {
            k0 = ws + (int64_t)(t - nsink) * T64;
            k1 = q_end;
        }
        if (k1 > k0 + T64) k1 = k0 + T64;
    }
};

__global__ void __launch_bounds__(NT, 2) win_fwd_kernel(const WinArgs a) {
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *kv = sq + TILE_F, *sp = kv + 4 * TILE_F;  // kv: K and V of two tiles
    const int64_t tiles = (a.N + T64 - 1) / T64;
    const int64_t q0 = (blockIdx.x % tiles) * T64;
    const int64_t bh = blockIdx.x / tiles;
    const int b = (int)(bh / a.H), h = (int)(bh % a.H), hk = h / a.G, half = a.r / 2;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    load_tile(sq, a.q.at<const float>(b, h, 0), a.q.sn, q0, a.N);
    __syncthreads();
    if (half) rotate_tile(sq, q0, a.N, a.rope, half, 1.f);
    float m[4], l[4], o[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int x = 0; x < 4; ++x) o[i][x] = 0.f;
    }
    const KeyTiles kt(q0, a.N, a.W, a.S);
    const float *kb = a.k.at<const float>(b, hk, 0), *vb = a.v.at<const float>(b, hk, 0);
    auto fetch = [&](int t) {
        int64_t k0, k1;
        kt.at(t, a.S, k0, k1);
        float* dst = kv + (t & 1) * 2 * TILE_F;
        fetch_tile(dst, kb, a.k.sn, k0, k1);
        fetch_tile(dst + TILE_F, vb, a.v.sn, k0, k1);
    };
    fetch(0);
    for (int t = 0; t < kt.n; ++t) {
        int64_t k0, k1;
        kt.at(t, a.S, k0, k1);
        float *sk = kv + (t & 1) * 2 * TILE_F, *sv = sk + TILE_F;
        landed();
        __syncthreads();
        if (t + 1 < kt.n) fetch(t + 1);  // beside this tile's work
        if (half) {
            rotate_tile(sk, k0, k1, a.rope, half, 1.f);
            __syncthreads();
        }
        float c[4][4];
        mm_nt(c, sq, sk, ty, tx);
        bool full = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t qi = q0 + ty + 16 * i;
            float mx = -INFINITY;
            bool seen[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t kj = k0 + tx + 16 * j;
                const bool ok = seen[j] = kj < k1 && visible(qi, kj, a.W, a.S);
                full = full && ok;
                c[i][j] = ok ? c[i][j] * a.scale_log2 : -INFINITY;
                mx = fmaxf(mx, c[i][j]);
            }
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float mn = fmaxf(m[i], mx);
            const float mz = mn == -INFINITY ? 0.f : mn;  // nothing seen yet
            const float al = exp2f(m[i] - mz);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float p = exp2f(c[i][j] - mz);
                sum += p;
                sp[(ty + 16 * i) * LD + tx + 16 * j] = seen[j] ? p : -0.f;
            }
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
            l[i] = l[i] * al + sum;
            m[i] = mn;
#pragma unroll
            for (int x = 0; x < 4; ++x) o[i][x] *= al;
        }
        full = __syncthreads_and(full);
        if (full)
            mm_nn<false>(o, sp, sv, ty, tx);
        else
            mm_nn<true>(o, sp, sv, ty, tx);
    }
    // every query sees itself: l > 0
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t qi = q0 + ty + 16 * i;
        if (qi >= a.N) continue;
        const float il = 1.f / l[i];
        *reinterpret_cast<float4*>(a.out.at<float>(b, h, qi) + 4 * tx) = make_float4(o[i][0] * il, o[i][1] * il, o[i][2] * il, o[i][3] * il);
        if (a.lse && tx == 0) a.lse[((int64_t)b * a.H + h) * a.N + qi] = m[i] + log2f(l[i]);
    }
}

// dq by query tiles; leaves D = dout . out in a.delta
__global__ void __launch_bounds__(NT, 2) win_dq_kernel(const WinArgs a) {
    extern __shared__ __align__(16) float sm[];
    float *sq = sm, *sdo = sq + TILE_F, *sv = sdo + TILE_F, *sds = sv + TILE_F, *ks = sds + TILE_F;  // ks: K of two tiles
    __shared__ float s_lse[T64], s_delta[T64];
    const int64_t tiles = (a.N + T64 - 1) / T64;
    const int64_t q0 = (blockIdx.x % tiles) * T64;
    const int64_t bh = blockIdx.x / tiles;
    const int b = (int)(bh / a.H), h = (int)(bh % a.H), hk = h / a.G, half = a.r / 2;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    load_tile(sq, a.q.at<const float>(b, h, 0), a.q.sn, q0, a.N);
    load_tile(sdo, a.dout.at<const float>(b, h, 0), a.dout.sn, q0, a.N);
    load_tile(sds, a.out.at<const float>(b, h, 0), a.out.sn, q0, a.N);
    __syncthreads();
    if (half) rotate_tile(sq, q0, a.N, a.rope, half, 1.f);
    {  // four threads a row
        const int row = threadIdx.x >> 2, part = threadIdx.x & 3;
        float s = 0.f;
        for (int x = part * 16; x < part * 16 + 16; ++x) s = fmaf(sdo[row * LD + x], sds[row * LD + x], s);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if (part == 0) {
            const int64_t at = bh * a.N + q0 + row;
            const bool in = q0 + row < a.N;
            s_delta[row] = s;
            s_lse[row] = in ? a.lse[at] : 0.f;
            if (in) a.delta[at] = s;
        }
    }
    float dq[4][4] = {};
    const KeyTiles kt(q0, a.N, a.W, a.S);
    const float *kb = a.k.at<const float>(b, hk, 0), *vb = a.v.at<const float>(b, hk, 0);
    auto fetch = [&](float* dst, const float* base, int64_t sn, int t) {
        int64_t k0, k1;
        kt.at(t, a.S, k0, k1);
        fetch_tile(dst, base, sn, k0, k1);
    };
    fetch(ks, kb, a.k.sn, 0);
    fetch(sv, vb, a.v.sn, 0);
    for (int t = 0; t < kt.n; ++t) {
        int64_t k0, k1;
        kt.at(t, a.S, k0, k1);
        float* sk = ks + (t & 1) * TILE_F;
        landed();
        __syncthreads();
        if (t + 1 < kt.n) fetch(ks + (~t & 1) * TILE_F, kb, a.k.sn, t + 1);  // beside this tile's work
        if (half) {
            rotate_tile(sk, k0, k1, a.rope, half, 1.f);
            __syncthreads();
        }
        float c[4][4], e[4][4];
        mm_nt(c, sq, sk, ty, tx);
        mm_nt(e, sdo, sv, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int qr = ty + 16 * i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t kj = k0 + tx + 16 * j;
                const bool ok = q0 + qr < a.N && kj < k1 && visible(q0 + qr, kj, a.W, a.S);
                const float p = ok ? exp2f(c[i][j] * a.scale_log2 - s_lse[qr]) : 0.f;
                sds[qr * LD + tx + 16 * j] = ok ? p * (e[i][j] - s_delta[qr]) : 0.f;
            }
        }
        __syncthreads();
        if (t + 1 < kt.n) fetch(sv, vb, a.v.sn, t + 1);  // (V is read no more)
        mm_nn<false>(dq, sds, sk, ty, tx);
    }
    __syncthreads();
    put_tile(sds, dq, [&](int i) { return ty + 16 * i; }, tx);
    __syncthreads();
    if (half) {
        rotate_tile(sds, q0, a.N, a.rope, half, -1.f);
        __syncthreads();
    }
    store_tile(sds, a.dq.at<float>(b, h, 0), a.dq.sn, q0, a.N, a.scale);
}

// dk and dv by key tiles: every query tile of the key head's G query heads whose window
// holds a key of the tile.  The queries behind that still see sinks (j < S) are further
// items, cut into parts of about a tile's own work; a part, and the first tiles where there
// are parts, leave the sinks' sums in scratch for win_sink_kernel.
struct DkvArgs {
    WinArgs a;
    int tiles, sink_tiles, parts, part_tiles;  // sink_tiles: key tiles with sinks; of each `parts` parts
    int64_t sink_q0;                           // first query of the parts
    float* part;                               // [B * Hkv][parts + 1][2][S][64]: dk', dv
};

__global__ void __launch_bounds__(NT, 2) win_dkv_kernel(const DkvArgs d) {
    extern __shared__ __align__(16) float sm[];
    float *sk = sm, *sv = sk + TILE_F, *sdo = sv + TILE_F, *sp = sdo + TILE_F, *qs = sp + TILE_F;  // qs: Q of two tiles
    __shared__ float s_lse[T64], s_delta[T64];
    const WinArgs& a = d.a;
    const int items = d.tiles + d.parts * d.sink_tiles;
    const int64_t bk = blockIdx.x / items;
    const int item = (int)(blockIdx.x % items), b = (int)(bk / a.Hkv), hk = (int)(bk % a.Hkv), half = a.r / 2;
    const bool sink = item >= d.tiles;
    const int pt = sink ? (item - d.tiles) / d.sink_tiles : 0;  // part of the sinks
    const int64_t k0 = (int64_t)(sink ? (item - d.tiles) % d.sink_tiles : item) * T64;
    const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
    load_tile(sk, a.k.at<const float>(b, hk, 0), a.k.sn, k0, a.N);
    load_tile(sv, a.v.at<const float>(b, hk, 0), a.v.sn, k0, a.N);
    __syncthreads();
    if (half) rotate_tile(sk, k0, a.N, a.rope, half, 1.f);
    float dk[4][4] = {}, dv[4][4] = {};
    // query tiles of a head, and of them all (head by head) the ones of this item
    const int64_t qb = sink ? d.sink_q0 : k0, qe = sink || k0 + T64 - 1 + a.W > a.N ? a.N : k0 + T64 - 1 + a.W;
    const int nq = (int)((qe - qb + T64 - 1) / T64), n0 = sink ? pt * d.part_tiles : 0;
    const int n1 = sink && n0 + d.part_tiles < nq * a.G ? n0 + d.part_tiles : nq * a.G;
    auto fetch = [&](float* dst, const Rows& x, int n) {
        fetch_tile(dst, x.at<const float>(b, hk * a.G + n / nq, 0), x.sn, qb + (int64_t)(n % nq) * T64, a.N);
    };
    if (n0 < n1) {
        fetch(qs, a.q, n0);
        fetch(sdo, a.dout, n0);
    }
    for (int n = n0; n < n1; ++n) {
        const int64_t q0 = qb + (int64_t)(n % nq) * T64, row = ((int64_t)b * a.H + hk * a.G + n / nq) * a.N;
        float* sq = qs + ((n - n0) & 1) * TILE_F;
        landed();
        __syncthreads();  // (and the last tile's rows of lse, delta and dS are read no more)
        if (n + 1 < n1) fetch(qs + (~(n - n0) & 1) * TILE_F, a.q, n + 1);  // beside this tile's work
        if (threadIdx.x < T64 && q0 + threadIdx.x < a.N) {
            s_lse[threadIdx.x] = a.lse[row + q0 + threadIdx.x];
            s_delta[threadIdx.x] = a.delta[row + q0 + threadIdx.x];
        }
        if (half) rotate_tile(sq, q0, a.N, a.rope, half, 1.f);
        __syncthreads();
        float c[4][4], e[4][4];
        mm_nt(c, sq, sk, ty, tx);
        mm_nt(e, sdo, sv, ty, tx);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int qr = ty + 16 * i;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t kj = k0 + tx + 16 * j, qi = q0 + qr;
                const bool ok = qi < a.N && (sink ? kj < a.S && qi - kj >= a.W : kj <= qi && qi - kj < a.W);
                const float p = ok ? exp2f(c[i][j] * a.scale_log2 - s_lse[qr]) : 0.f;
                sp[qr * LD + tx + 16 * j] = p;
                e[i][j] = ok ? p * (e[i][j] - s_delta[qr]) : 0.f;
            }
        }
        __syncthreads();
        mm_tn(dv, sp, sdo, ty, tx);
        __syncthreads();
        if (n + 1 < n1) fetch(sdo, a.dout, n + 1);  // (dO is read no more, and dS takes P's place)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sp[(ty + 16 * i) * LD + tx + 16 * j] = e[i][j];
        __syncthreads();
        mm_tn(dk, sp, sq, ty, tx);
    }
    __syncthreads();
    if (d.parts && k0 < a.S) {
        float* part = d.part + (bk * (d.parts + 1) + (sink ? pt + 1 : 0)) * 2 * a.S * D;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t j = k0 + 4 * ty + i;
            if (j >= a.S) continue;
            *reinterpret_cast<float4*>(part + j * D + 4 * tx) = make_float4(dk[i][0], dk[i][1], dk[i][2], dk[i][3]);
            *reinterpret_cast<float4*>(part + (a.S + j) * D + 4 * tx) = make_float4(dv[i][0], dv[i][1], dv[i][2], dv[i][3]);
        }
        if (sink) return;
    }
    put_tile(sp, dv, [&](int i) { return 4 * ty + i; }, tx);
    put_tile(qs, dk, [&](int i) { return 4 * ty + i; }, tx);
    __syncthreads();
    if (half) {
        rotate_tile(qs, k0, a.N, a.rope, half, -1.f);
        __syncthreads();
    }
    store_tile(sp, a.dv.at<float>(b, hk, 0), a.dv.sn, k0, a.N, 1.f);
    store_tile(qs, a.dk.at<float>(b, hk, 0), a.dk.sn, k0, a.N, a.scale);
}

cudaError_t fwd(const WinArgs& a, cudaStream_t s) {
    const int smem = 6 * TILE_F * 4;
    cudaError_t e = allow_smem<win_fwd_kernel>(smem);
    if (e != cudaSuccess) return e;
    const int64_t grid = (a.N + T64 - 1) / T64 * a.B * a.H;
    win_fwd_kernel<<<(unsigned)grid, NT, smem, s>>>(a);
    return cudaGetLastError();
}
cudaError_t bwd(const WinArgs& a, void* scratch, cudaStream_t s) {
    const int sm_q = 6 * TILE_F * 4, sm_kv = 6 * TILE_F * 4;
    cudaError_t e = allow_smem<win_dq_kernel>(sm_q);
    if (e == cudaSuccess) e = allow_smem<win_dkv_kernel>(sm_kv);
    if (e != cudaSuccess) return e;
    const WinSimtPlan pl = win_simt_plan(a);
    DkvArgs d{};
    d.a = a;
    d.a.delta = static_cast<float*>(scratch);
    d.tiles = (int)((a.N + T64 - 1) / T64);
    d.sink_tiles = pl.parts ? (a.S + T64 - 1) / T64 : 1;
    d.parts = pl.parts;
    d.part_tiles = pl.part_tiles;
    d.sink_q0 = pl.sink_q0;
    d.part = reinterpret_cast<float*>(static_cast<char*>(scratch) + pl.part);
    win_dq_kernel<<<(unsigned)((int64_t)d.tiles * a.B * a.H), NT, sm_q, s>>>(d.a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    win_dkv_kernel<<<(unsigned)((int64_t)(d.tiles + d.parts * d.sink_tiles) * a.B * a.Hkv), NT, sm_kv, s>>>(d);
    e = cudaGetLastError();
    if (e != cudaSuccess || !d.parts) return e;
    return launch_win_sinks(a, d.part, d.parts, false, s);
}

}  // namespace wins

WinSimtPlan win_simt_plan(const WinArgs& a) {
    WinSimtPlan p{};
    if (a.S > 0 && a.N > a.W) {
        p.sink_q0 = a.W / 64 * 64;
        const int64_t all = (a.N - p.sink_q0 + 63) / 64 * a.G;
        int64_t per = (int64_t)a.G * ((a.W + 126) / 64 + 1);  // a key tile's own
        if (all > per * 256) per = (all + 255) / 256;
        p.part_tiles = (int)per;
        p.parts = (int)((all + per - 1) / per);
    }
    p.part = ((size_t)a.B * a.H * a.N * 4 + 255) / 256 * 256;  // behind dout . out per query
    p.total = p.part + (p.parts ? (size_t)a.B * a.Hkv * (p.parts + 1) * 2 * a.S * D * 4 : 0);
    return p;
}

cudaError_t launch_win_fwd_simt(const WinArgs& a, cudaStream_t s) { return wins::fwd(a, s); }
cudaError_t launch_win_bwd_simt(const WinArgs& a, void* scratch, cudaStream_t s) { return wins::bwd(a, scratch, s); }

}  // namespace kvm
