// Attention of the newest tokens over the paged cache (decode).
//
//   out = sum_j softmax_j(q' . k_j / 8) v_j over j <= p and (W == 0 or p - j < W or j < S)
//
// Bound by the visible cache rows, each read once: the R = G T query rows of a key
// head (16, or 32 at once) share every row that is loaded.
//
// The work is a list of steps of 32 keys, item by item (an item: one sequence, key head
// and tile of query rows); every computing warp of the grid takes an equal, contiguous
// part of it, whatever the lengths are.  The lengths are read on the device, so a
// captured call serves growing sequences.  One CTA per SM: four loading warps fill a ring
// in shared memory for each computing warp (a group of eight lanes serves one ring, a
// lane one run of the step's rows that lie together in a page: TMA tiles, or bulk copies
// for the 4-bit rows; page indexes are fetched two steps ahead), so the computing warps
// only wait, multiply and release.  With the loads in the computing warps themselves a
// step cost them about as long again.  An item inside one warp's part is written at once;
// parts of an item split over warps go to scratch and are joined by a second kernel in
// the order of the warps, so results do not depend on timing.  The grid is this card's 152
// SMs whatever part of them a call gets, as the scratch's size and the sums' order follow it.
//
// Queries of one sequence see nearly the same keys.  The few that only some of them see are
// looked at when they come by; where their value is not finite, it stays out of the products
// and is added row by row (four queries a sequence: 1 to 2% of a call, 6% of 64 short windows).
//
// bf16 pages: mma.sync m16n8k16 with fp32 sums, K and V fragments by 16-byte shared
// loads (dims and tokens are permuted alike on both sides of each product, which lets a
// thread's operands lie next to one another).  The tensor cores are not what bounds
// this kernel: a step of 8 KB takes 32 of these products, 64 cycles of the tensor core
// beside 348 of its share of the memory.
// 4-bit pages: codes become bf16 128 + c by one logic operation for two; a row's scale
// and least value enter the score, where the offset leaves too (128 sum q), and for the
// values the probability.  Values are centred, c - 8, before their product: the offset
// taken from the sums at the end would leave errors of sums 130 times the result's size
// (at 65,536 keys 0.8% of the result).
// Up to 8 query rows in 4 bits change places with the keys (S^T = K Q^T, O^T += V^T P^T, P^T
// through movmatrix): half the products, and no exponentials for rows that are not there
// (57.5 to 51.2 us for the same sequences; the rest is unpacking, which does not shrink).
// fp32: the same walk with fp32 multiply-adds, a lane a key for the scores and two dims
// a lane for the sum: 152 us for 24 sequences to 16,000 keys, 16 heads of 4 (3.9 TB/s), 6.6
// TB/s with a row a key head (64 sequences of 16,384 keys, 8 heads).  Bound by those with more rows; latencies count, so eight warps
// of one stage (four of three: half as fast), short chains, four keys' probabilities a load.
#include "kvm_paged.cuh"
#include "tc_primitives.cuh"

namespace kvm {
namespace {

using tc::ex2;
using tc::smem_u32;

constexpr int NLOAD = 4;       // loading warps
constexpr int KS = 32;         // keys per step
constexpr int MIN_STEPS = 4;   // fewest steps worth a warp of their own
constexpr int NSM = 152;       // CTAs
constexpr int MAX_PRE = 256;   // sequences whose first steps a CTA keeps

enum { F_BF16 = 0, F_I4 = 1, F_FP32 = 2, F_I4_FP32 = 3 };

template <int F, int MT> struct Cfg {
    static constexpr bool I4 = F == F_I4 || F == F_I4_FP32;
    static constexpr bool MMA = F == F_BF16 || F == F_I4;
    static constexpr bool SWAP = MMA && MT == 0;  // up to 8 query rows, as the products' columns
    static constexpr int M = SWAP ? 1 : MT;
    using T = typename std::conditional<MMA, __nv_bfloat16, float>::type;
    static constexpr int RB = I4 ? 32 : (F == F_BF16 ? 128 : 256);  // bytes of a cached row
    static constexpr int SMO = 2 * KS * RB;                         // offset of the scales in a stage
    static constexpr int STAGE = SMO + (I4 ? 2 * KS * 4 : 0);
    static constexpr int STAGES = SWAP ? 5 : I4 ? 6 : F == F_FP32 ? 1 : 3;
    static constexpr int ROWS = SWAP ? 8 : 16 * MT;                 // query rows at once
    // computing warps: what the registers (4 bits: 104 and 152 a thread) and the rings leave room for;
    // SWAP with 12: 51.2 us where 16 take 49.0 (8 sequences to 65,536 keys, 16 heads of 4, one token)
    static constexpr int NC = SWAP ? 16 : F == F_I4 && MT == 1 ? 12 : 8;
    static constexpr int THREADS = 32 * (NLOAD + NC);
    // register split of the launch's registers (multiples of 8, 65536 / THREADS a thread at most)
    static constexpr int REGS_LOAD = NC == 12 ? 56 : 40, REGS = NC == 16 ? 104 : NC == 12 ? 152 : 232;
    static constexpr int QB = MMA ? ROWS * 128 : ROWS * 256 + ROWS * KS * 4;  // q (and fp32: p) of a warp
    static constexpr int RING = I4 ? QB : (QB + 1023) / 1024 * 1024;          // swizzled tiles lie on 1024 bytes
    static constexpr int WARP = RING + STAGES * STAGE;
    static constexpr int BARS = NC * WARP;                          // full, empty barriers and a word per stage
    static constexpr int SMEM = BARS + NC * STAGES * 24 + 16 + (1 + MAX_PRE) * 4 + 1024;
    static_assert(SMEM <= 227 * 1024, "shared memory of a CTA");
};

struct Plan {
    int rows;      // query rows of a tile
    int tiles;     // of the R rows of a key head
    int warps;
    size_t slot;   // floats of a part
};
template <int F, int MT> Plan plan_for(int R) {
    using C = Cfg<F, MT>;
    Plan p;
    p.tiles = (R + C::ROWS - 1) / C::ROWS;
    p.rows = (R + p.tiles - 1) / p.tiles;
    p.warps = C::NC * NSM;
    p.slot = (size_t)p.rows * (D + 2);
    return p;
}

struct AttnP {
    PagedArgs a;
    int* first;  // scratch: steps (of one item each) before every sequence, and all [B + 1]
    FastDiv by_t, by_half;
    Plan pl;
    int R;
    uint32_t all_runs;  // bits of a step's runs
    int run, run_bits;  // rows of a step that lie together: min(page_size, 32)
};

// What sequence b's queries see, in steps of 32 keys at multiples of 32: `sink` steps from
// key 0, then from `from` on.
struct Span {
    int len;
    int from, sink, steps;
    int oldest;  // position of query t = 0 (negative where len < T)
    __device__ __forceinline__ void of(const PagedArgs& a, int b, bool report) {
        len = a.lens[b];
        if (len < 0 || len > a.cap) {
            if (report && a.status) atomicOr(a.status, KVM_DEV_DATA);
            len = len < 0 ? 0 : (int)a.cap;
        }
        oldest = len - a.T;
        const int first = max(oldest, 0), ws = a.W > 0 ? max(first - a.W + 1, 0) : 0;  // (W < 2^31: no overflow)
        from = ws & ~(KS - 1);
        sink = (min(a.S, ws) + KS - 1) / KS;
        if (sink * KS >= from) sink = from = 0;  // (they meet)
        steps = sink + (len - from + KS - 1) / KS;
        if (steps < 1) steps = 1;  // (nothing cached: the step that writes zeros)
    }
    __device__ __forceinline__ int base(int step) const { return step < sink ? KS * step : from + KS * (step - sink); }
};

// Steps of all sequences (of one item each), by one warp; those before each also to pre
// (shared, up to MAX_PRE sequences) and out (scratch) where these are not null.
__device__ __forceinline__ int all_steps(const PagedArgs& a, int lane, int* pre, int* out) {
    int done = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int b = b0 + lane;
        int n = 0;
        if (b < a.B) {
            Span s;
            s.of(a, b, false);
            n = s.steps;
        }
        int up = n;  // inclusive scan
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up += y;
        }
        if (b < a.B) {
            if (pre) pre[b] = done + up - n;
            if (out) out[b] = done + up - n;
        }
        done += __shfl_sync(0xffffffffu, up, 31);
    }
    if (lane == 0 && out) out[a.B] = done;
    return done;
}
// The sequence that step `at` of the list falls in, and that sequence's first step.
// (for more than MAX_PRE sequences)
__device__ __forceinline__ void find_sequence(const PagedArgs& a, int items, int at, int lane, int& b, int& first) {
    int done = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        int n = 0;
        if (b0 + lane < a.B) {
            Span s;
            s.of(a, b0 + lane, false);
            n = s.steps * items;
        }
        int up = n;  // inclusive scan
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, up, o);
            if (lane >= o) up += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, done + up > at);
        if (past) {
            const int w = __ffs(past) - 1;
            b = b0 + w;
            first = done + __shfl_sync(0xffffffffu, up - n, w);
            return;
        }
        done += __shfl_sync(0xffffffffu, up, 31);
    }
    b = a.B;
    first = done;
}
// The parts: the first `more` of n warps take per + 1 steps, the others per.
struct Parts {
    int n, per, more;
    __device__ __forceinline__ Parts(int total, int warps) {
        n = max(1, min(total / MIN_STEPS, warps));
        per = total / n;
        more = total - per * n;
    }
    __device__ __forceinline__ int begin(int w) const { return w * per + min(w, more); }
    __device__ __forceinline__ int of(int step) const {
        const int m = more * (per + 1);
        return step < m ? step / (per + 1) : more + (step - m) / per;
    }
};

// position in the list of steps
struct Walk {
    int b, hk, tile, step;
    Span s;
    __device__ __forceinline__ void next(const PagedArgs& a, int tiles, bool report) {
        if (++step < s.steps) return;
        step = 0;
        if (++tile < tiles) return;
        tile = 0;
        if (++hk < a.Hkv) return;
        hk = 0;
        if (++b < a.B) s.of(a, b, report);
    }
};

// bulk copy (16-byte aligned, a multiple of 16 bytes) and tile copy of 64 bf16 dims, completing on a barrier
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int x, int row, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(row), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// (the same from zero)
__device__ __forceinline__ void mma16816_0(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
                 "{%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// an 8 x 8 tile of 16-bit values, a row's pairs over four lanes, transposed
__device__ __forceinline__ uint32_t transposed(uint32_t a) {
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&h);
}
// two bf16 128 + c -> c - 8 (exact)
__device__ __forceinline__ uint32_t centred(uint32_t w) {
    const uint32_t k = 0x43084308u;  // 136
    const __nv_bfloat162 y = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&k));
    return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ bool sees(const PagedArgs& a, int p, int j) {
    return j <= p && (a.W == 0 || p - j < a.W || j < a.S);
}

// some half of a word of two bf16, or a word that is an fp32 value, is not finite
template <typename T> __device__ __forceinline__ bool odd_word(uint32_t w) {
    return (w & 0x7f800000u) == 0x7f800000u || (sizeof(T) == 2 && (w & 0x7f80u) == 0x7f80u);
}

template <int F, int MT>
__global__ void __launch_bounds__(Cfg<F, MT>::THREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const __grid_constant__ AttnP ap) {
    using C = Cfg<F, MT>;
    using T = typename C::T;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* const smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const PagedArgs& a = ap.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int tiles = ap.pl.tiles, rows = ap.pl.rows, items = a.Hkv * tiles;
    const uint32_t bars = smem_u32(smem + C::BARS);
    auto full = [&](int ring, int st) { return bars + 8 * (ring * C::STAGES + st); };
    auto empty = [&](int ring, int st) { return bars + 8 * ((C::NC + ring) * C::STAGES + st); };
    volatile uint32_t* const good = reinterpret_cast<volatile uint32_t*>(smem + C::BARS + C::NC * C::STAGES * 16);  // runs copied
    volatile int* const abort_flag = reinterpret_cast<volatile int*>(smem + C::BARS + C::NC * C::STAGES * 24);
    for (int i = threadIdx.x; i < 2 * C::NC * C::STAGES; i += C::THREADS) tc::mbar_init(bars + 8 * i, 1);
    if (threadIdx.x == 0) *abort_flag = 0;
    tc::fence_barrier_init();
    tc::fence_proxy_async();
    int* const pre = reinterpret_cast<int*>(smem + C::BARS + C::NC * C::STAGES * 24 + 16);
    if (warp == 0) {
        const int n = all_steps(a, lane, a.B <= MAX_PRE ? pre + 1 : nullptr, blockIdx.x == 0 ? ap.first : nullptr);
        if (lane == 0) pre[0] = n;
    }
    __syncthreads();
    const int total = pre[0] * items;
    const Parts parts(total, ap.pl.warps);

    // the warps of one SM lie next to one another in the list only by chance of the lengths: warp w of
    // CTA x is worker w * gridDim.x + x, so that few workers fill few SMs' loaders alike
    auto worker = [&](int w) { return w * (int)gridDim.x + (int)blockIdx.x; };
    auto start = [&](int at, Walk& w) {
        int first;
        if (a.B <= MAX_PRE) {  // the last sequence that begins at or before the step
            int lo = 0, hi = a.B - 1;
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (pre[1 + mid] * items <= at)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            w.b = lo;
            first = pre[1 + lo] * items;
        } else {
            find_sequence(a, items, at, lane, w.b, first);
        }
        w.s.of(a, w.b, lane == 0);
        const int in = at - first, item = in / w.s.steps;
        w.step = in - item * w.s.steps;
        w.hk = item / tiles;
        w.tile = item - w.hk * tiles;
    };
    // some query sees key j
    auto wanted = [&](const Span& s, int j) { return j < s.len && (a.W == 0 || max(s.oldest, 0) - j < a.W || j < a.S); };

    if (warp < NLOAD) {
        // ------------------------------------------------------------- loading
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_LOAD));
        constexpr int RINGS = C::NC / NLOAD;  // of this warp: eight lanes each
        const int grp = lane >> 3, r = lane & 7, lead = lane & ~7;
        const int ring = grp * NLOAD + warp;
        Walk w{};
        int count = 0;
        auto take = [&](int i) {
            const int gw = worker(i * NLOAD + warp);
            if (gw >= parts.n) return;
            Walk x;
            const int at = parts.begin(gw);
            start(at, x);
            if (grp == i) {
                w = x;
                count = parts.begin(gw + 1) - at;
            }
        };
        if (a.B <= MAX_PRE) {  // each group looks for its own
            if (grp < RINGS) take(grp);
            __syncwarp();
        } else {
#pragma unroll 1
            for (int i = 0; i < RINGS; ++i) take(i);
        }
        const uint32_t ring_s = smem_u32(smem + ring * C::WARP + C::RING);
        const uint8_t *pk = reinterpret_cast<const uint8_t*>(a.k), *pv = reinterpret_cast<const uint8_t*>(a.v);
        // this lane's run of the next step: its page index (only read here: the latency passes behind
        // two steps) and where its rows lie in a page, -1 when no query sees a key of it
        int seen = 0;  // steps looked up
        auto look_up = [&](int& pg, int& in_page) {
            in_page = -1;
            if (seen >= count) return;
            const int j = w.s.base(w.step) + r * ap.run;
            // (a run holds a key that is seen: its last key in the window, or its first among the sinks)
            if (r * ap.run < KS && j < w.s.len && (wanted(w.s, min(j + ap.run, w.s.len) - 1) || wanted(w.s, j))) {
                in_page = (w.hk << a.page_bits) + (j & (a.page_size - 1));
                pg = a.table[(int64_t)w.b * a.max_pages + (j >> a.page_bits)];
            }
            if (++seen < count) w.next(a, tiles, r == 0);
        };
        int pg0 = 0, in0 = -1, pg1 = 0, in1 = -1;
        look_up(pg0, in0);
        look_up(pg1, in1);
        int done = 0, st = 0;
        uint32_t phase = 1;  // (an empty ring's barriers count as released)
        long long t0 = clock64();
        while (__any_sync(0xffffffffu, done < count)) {
            bool ready = done < count && r == 0 && tc::mbar_try(empty(ring, st), phase);
            ready = __shfl_sync(0xffffffffu, ready, lead);
            if (!__any_sync(0xffffffffu, ready)) {
                if (__any_sync(0xffffffffu, *abort_flag || clock64() - t0 > (1ll << 33))) break;  // (the computing warps report)
                continue;
            }
            t0 = clock64();
            const bool there = pg0 >= 0 && pg0 < a.n_pages, ok = ready && in0 >= 0 && there;
            if (ready && in0 >= 0 && !there && a.status) atomicOr(a.status, KVM_DEV_DATA);
            const uint32_t runs = (__ballot_sync(0xffffffffu, ok) >> lead) & 0xff;
            const uint32_t bar = full(ring, st), base = ring_s + st * C::STAGE, at = r * ap.run;
            if (ready && r == 0) {
                good[ring * C::STAGES + st] = runs;
                tc::mbar_expect_tx(bar, __popc(runs) * ap.run * (C::STAGE / KS));
            }
            __syncwarp();
            if (ok) {
                const int64_t row = (((int64_t)pg0 * a.Hkv) << a.page_bits) + in0;
                if constexpr (F == F_BF16) {
                    tma_rows(base + at * 128, &tm_k, 0, (int)row, bar);
                    tma_rows(base + KS * 128 + at * 128, &tm_v, 0, (int)row, bar);
                } else if constexpr (F == F_FP32) {  // two halves of 32 dims
                    tma_rows(base + at * 128, &tm_k, 0, (int)row, bar);
                    tma_rows(base + KS * 128 + at * 128, &tm_k, 32, (int)row, bar);
                    tma_rows(base + KS * 256 + at * 128, &tm_v, 0, (int)row, bar);
                    tma_rows(base + KS * 384 + at * 128, &tm_v, 32, (int)row, bar);
                } else {
                    const uint32_t n = ap.run * C::RB, ns = ap.run * 4;
                    bulk_load(base + at * C::RB, pk + row * C::RB, n, bar);
                    bulk_load(base + KS * C::RB + at * C::RB, pv + row * C::RB, n, bar);
                    bulk_load(base + C::SMO + at * 4, a.k_sm + row, ns, bar);
                    bulk_load(base + C::SMO + KS * 4 + at * 4, a.v_sm + row, ns, bar);
                }
            }
            __syncwarp();
            if (ready) {
                pg0 = pg1;
                in0 = in1;
                look_up(pg1, in1);
                ++done;
                if (++st == C::STAGES) st = 0, phase ^= 1;
            }
        }
        if (*abort_flag) {  // let the copies issued last land before the CTA ends
            for (int x = 0; x < C::STAGES && x < done; ++x) {
                if (--st < 0) st = C::STAGES - 1, phase ^= 1;
                const long long t1 = clock64();
                while (!tc::mbar_try(full(ring, st), phase ^ 1) && clock64() - t1 < (1ll << 28)) {
                }
            }
        }
        return;
    }

    // --------------------------------------------------------------- computing
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS));
    const int ring_id = warp - NLOAD, gw = worker(ring_id);
    if (gw >= parts.n) return;
    const int begin = parts.begin(gw), count = parts.begin(gw + 1) - begin;
    uint8_t* const sq = smem + ring_id * C::WARP;
    uint8_t* const ring = sq + C::RING;
    Walk cp;
    start(begin, cp);

    const int g = lane >> 2, c = lane & 3;
    // column n of a tile of 8 keys is its key tk(n): tk(2 c) = c, tk(2 c + 1) = 4 + (c + 2) % 4 (no two
    // lanes of a shared load then meet in a bank); ka, kb: this lane's columns, tk of column g for K
    const int ka = c, kb = 4 + ((c + 2) & 3), tg = (g & 1) ? 4 + (((g >> 1) + 2) & 3) : g >> 1;
    const int off_k = F == F_BF16 ? tg * 128 + ((c ^ tg) << 4) : tg * 32 + c * 8;
    const int off_a = F == F_BF16 ? ka * 128 + ((g ^ ka) << 4) : ka * 32 + g * 4;
    const int off_b = F == F_BF16 ? kb * 128 + ((g ^ kb) << 4) : kb * 32 + g * 4;
    // tensor-core state: query fragments, sums; O[mt][nt]: rows g, g + 8, dims 16 c + nt and 16 c + 8 + nt
    // SWAP: keys (scores) and dims (values) are the products' rows, queries 2 c, 2 c + 1 this lane's
    // columns; O[0][w]: dims 8 g + 2 w and 8 g + 2 w + 1 of both
    constexpr int M = C::M;
    uint32_t qf[C::MMA ? M : 1][4][4];
    float O[C::MMA ? M : 1][8][4];
    float qsum[M][2], vmin[M][2];
    float m[C::MMA ? 2 * M : 16], l[C::MMA ? 2 * M : 16];
    float acc[C::MMA ? 1 : 16][2];
    bool fresh = true;
    int seg = 0;
    int st = 0;
    uint32_t phase = 0;

    int nr = 0, r0 = 0;           // query rows of the item: nr from r0 of its key head's
    int pos[C::MMA ? 2 * M : 1];  // positions of this lane's rows (-1: no row)

    for (int at = 0; at < count; ++at) {
        const int hk = cp.hk;
        if (fresh) {
            fresh = false;
            seg = at;
            r0 = cp.tile * rows;
            nr = min(rows, ap.R - r0);
            // the item's query rows into this warp's shared memory, rows past them zero, all loads at
            // once; then their rotation, a pair of dims a lane
            __syncwarp();
            constexpr int PCS = D * (int)sizeof(T) / 16;  // 16-byte pieces of a row
#pragma unroll
            for (int i = 0; i < C::ROWS * PCS / 32; ++i) {
                const int x = i * 32 + lane, r = x / PCS, gt = r0 + r, gh = ap.by_t.div(gt);
                uint4 y = make_uint4(0, 0, 0, 0);
                if (r < nr) y = reinterpret_cast<const uint4*>(a.q.at<const T>(cp.b, hk * a.G + gh, gt - gh * a.T))[x % PCS];
                reinterpret_cast<uint4*>(sq)[x] = y;
            }
            __syncwarp();
            if (const int half = a.r / 2; half > 0) {
#pragma unroll 4
                for (int x = lane; x < nr * half; x += 32) {
                    const int r = ap.by_half.div(x), d = x - r * half, gt = r0 + r, p = cp.s.oldest + gt - ap.by_t.div(gt) * a.T;
                    if (p < 0) continue;  // (sees nothing)
                    const float2 cs = a.rope[(int64_t)p * half + d];
                    T* y = reinterpret_cast<T*>(sq) + r * D + d;
                    const float u = to_f<T>(y[0]), v = to_f<T>(y[half]);
                    y[0] = from_f<T>(u * cs.x - v * cs.y);
                    y[half] = from_f<T>(v * cs.x + u * cs.y);
                }
                __syncwarp();
            }
            if constexpr (C::SWAP) {
                const uint16_t* qu = reinterpret_cast<const uint16_t*>(sq) + g * D;
                float s = 0.f;
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int d = 16 * c + 8 * (ks >> 1) + 2 * (ks & 1) + x;
                        const uint32_t w = (uint32_t)qu[d] | ((uint32_t)qu[d + 4] << 16);
                        qf[0][ks][x] = w;
                        s += lo_f(w) + hi_f(w);
                    }
                s += __shfl_xor_sync(0xffffffffu, s, 1);
                s += __shfl_xor_sync(0xffffffffu, s, 2);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 2 * c + e;
                    qsum[0][e] = __shfl_sync(0xffffffffu, s, 4 * r);
                    vmin[0][e] = l[e] = 0.f;
                    m[e] = -INFINITY;
                    pos[e] = r < nr ? cp.s.oldest + r0 + r - ap.by_t.div(r0 + r) * a.T : -1;
                }
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int x = 0; x < 4; ++x) O[0][w][x] = 0.f;
            } else if constexpr (C::MMA) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const __nv_bfloat16* qr = reinterpret_cast<const __nv_bfloat16*>(sq) + (mt * 16 + g + 8 * u) * D;
                        if constexpr (F == F_BF16) {
                            // k-steps 0, 1: dims 8 c ..; 2, 3: dims 32 + 8 c ..
#pragma unroll
                            for (int hf = 0; hf < 2; ++hf) {
                                const uint4 x = *reinterpret_cast<const uint4*>(qr + 32 * hf + 8 * c);
                                qf[mt][2 * hf][u] = x.x;
                                qf[mt][2 * hf][2 + u] = x.y;
                                qf[mt][2 * hf + 1][u] = x.z;
                                qf[mt][2 * hf + 1][2 + u] = x.w;
                            }
                        } else {
                            // a word of codes holds dims d .. d + 7: pairs (d, d + 4), (d + 1, d + 5), ..
                            const uint16_t* qu = reinterpret_cast<const uint16_t*>(qr);
                            float s = 0.f;
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                                for (int x = 0; x < 2; ++x) {
                                    const int d = 16 * c + 8 * (ks >> 1) + 2 * (ks & 1) + x;
                                    const uint32_t w = (uint32_t)qu[d] | ((uint32_t)qu[d + 4] << 16);
                                    qf[mt][ks][2 * x + u] = w;
                                    s += lo_f(w) + hi_f(w);
                                }
                            s += __shfl_xor_sync(0xffffffffu, s, 1);
                            s += __shfl_xor_sync(0xffffffffu, s, 2);
                            qsum[mt][u] = s;
                            vmin[mt][u] = 0.f;
                        }
                        m[2 * mt + u] = -INFINITY;
                        l[2 * mt + u] = 0.f;
                        const int r = mt * 16 + g + 8 * u;
                        pos[2 * mt + u] = r < nr ? cp.s.oldest + r0 + r - ap.by_t.div(r0 + r) * a.T : -1;
                    }
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
#pragma unroll
                        for (int nt = 0; nt < 8; ++nt) O[mt][nt][x] = 0.f;
                    }
                }
            } else {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    m[r] = -INFINITY;
                    l[r] = acc[r][0] = acc[r][1] = 0.f;
                }
            }
        }
        if (!tc::mbar_wait_warp(full(ring_id, st), phase, abort_flag, a.status)) {
            for (int x = 0; x < C::STAGES && at + x < count; ++x) {  // (copies under way land first)
                const long long t1 = clock64();
                while (!tc::mbar_try(full(ring_id, st), phase) && clock64() - t1 < (1ll << 26)) {
                }
                if (++st == C::STAGES) st = 0, phase ^= 1;
            }
            return;
        }
        const uint8_t* sk = ring + st * C::STAGE;
        const uint8_t* sv = sk + KS * C::RB;
        const int base = cp.s.base(cp.step);
        const int oldest = cp.s.oldest;
        // keep: keys that some query sees and whose page exists; whole: every row sees every key
        uint32_t keep = good[ring_id * C::STAGES + st];
        bool whole = oldest >= base + KS - 1 && (a.W == 0 || cp.s.len - 1 - base < a.W || base + KS <= a.S);
        // alone: keys that some queries see and others do not (the newest of a.T tokens, and with a
        // window the first) whose value is not finite.  A product would carry it to the others, as
        // 0 x NaN is NaN: their values are left out of it and reach the rows that see them apart.
        uint32_t alone = 0;
        if (!whole || keep != ap.all_runs) {
            whole = false;
            const int j = base + lane;
            const bool in = ((keep >> (lane >> ap.run_bits)) & 1) && wanted(cp.s, j);
            keep = __ballot_sync(0xffffffffu, in);
            if (a.T > 1) {
                const bool part = in && !(j <= oldest && (a.W == 0 || cp.s.len - 1 - j < a.W || j < a.S));
                if (__any_sync(0xffffffffu, part)) {
                    bool odd = false;
                    if constexpr (C::I4) {
                        odd = odd_word<__nv_bfloat16>(*reinterpret_cast<const uint32_t*>(sk + C::SMO + (KS + lane) * 4));
                    } else {
#pragma unroll
                        for (int x = 0; x < C::RB / 16; ++x) {
                            const uint4 y = *reinterpret_cast<const uint4*>(sv + (x >> 3) * KS * 128 + lane * 128 + (((x & 7) ^ (lane & 7)) << 4));
                            odd = odd || odd_word<T>(y.x) || odd_word<T>(y.y) || odd_word<T>(y.z) || odd_word<T>(y.w);
                        }
                    }
                    alone = __ballot_sync(0xffffffffu, part && odd);
                }
            }
        } else {
            keep = ~0u;
        }

        if constexpr (C::SWAP) {
            // S^T = K Q^T of two tiles of 8 keys at once: S[i][e], S[i][2 + e]: this lane's key tg of
            // tiles 2 i and 2 i + 1, its query e
            float S[2][4];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t kf[2][8];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint2 w = *reinterpret_cast<const uint2*>(sk + 256 * (2 * i + x) + off_k);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        kf[x][y] = ((w.x >> (4 * y)) & 0x000f000fu) | 0x43004300u;
                        kf[x][4 + y] = ((w.y >> (4 * y)) & 0x000f000fu) | 0x43004300u;
                    }
                }
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    const uint32_t A[4] = {kf[0][2 * ks], kf[1][2 * ks], kf[0][2 * ks + 1], kf[1][2 * ks + 1]};
                    if (ks == 0)
                        mma16816_0(S[i], A, qf[0][ks][0], qf[0][ks][1]);
                    else
                        mma16816(S[i], A, qf[0][ks][0], qf[0][ks][1]);
                }
            }
            const uint32_t* ps = reinterpret_cast<const uint32_t*>(sk + C::SMO);
            uint32_t ksm[4], vsm[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                ksm[j] = ps[8 * j + tg];
                vsm[j] = ps[KS + 8 * j + tg];
            }
            if (!whole) {  // scales of keys that are not there may be anything
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = 8 * j + tg;
                    if (!((keep >> k) & 1)) ksm[j] = vsm[j] = 0;
                    if (alone >> k & 1) {  // (scale or least value is not finite: no dim of the row is)
                        vsm[j] = 0;
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (sees(a, pos[e], base + k)) vmin[0][e] = NAN;
                    }
                }
            }
            // (scale, least value and offset as below, two queries at once)
            float2 s2[4];
            const float2 qs = make_float2(qsum[0][0], qsum[0][1]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float sc = lo_f(ksm[j]), off = fmaf(sc, -128.f, hi_f(ksm[j]));
                s2[j] = __ffma2_rn(make_float2(S[j >> 1][2 * (j & 1)], S[j >> 1][2 * (j & 1) + 1]), make_float2(sc, sc),
                                   __fmul2_rn(make_float2(off, off), qs));
            }
            if (!whole) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int k = 8 * j + tg;
                    const bool in = (keep >> k) & 1;
                    if (!in || !sees(a, pos[0], base + k)) s2[j].x = -INFINITY;
                    if (!in || !sees(a, pos[1], base + k)) s2[j].y = -INFINITY;
                }
            }
            float2 mx = make_float2(tc::fmax3(fmaxf(s2[0].x, s2[1].x), s2[2].x, s2[3].x), tc::fmax3(fmaxf(s2[0].y, s2[1].y), s2[2].y, s2[3].y));
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                mx.x = fmaxf(mx.x, __shfl_xor_sync(0xffffffffu, mx.x, o));
                mx.y = fmaxf(mx.y, __shfl_xor_sync(0xffffffffu, mx.y, o));
            }
            // the maximum follows only when it grows by more than 2^8 (fp32 sums absorb that)
            float al[2] = {1.f, 1.f};
            bool grow = false;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float y = (e ? mx.y : mx.x) * a.scale_log2;
                if (y > m[e] + 8.f || (m[e] == -INFINITY && y > m[e])) {
                    al[e] = ex2(m[e] - y);
                    m[e] = y;
                    grow = true;
                }
            }
            const float2 sc2 = make_float2(a.scale_log2, a.scale_log2);
            const float2 mz2 = make_float2(m[0] == -INFINITY ? 0.f : -m[0], m[1] == -INFINITY ? 0.f : -m[1]);
            float2 sum = make_float2(0.f, 0.f), low = make_float2(0.f, 0.f);
            uint32_t P[4];  // [tile]: this lane's query g, the keys of columns 2 c, 2 c + 1
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = __ffma2_rn(s2[j], sc2, mz2);
                const float2 p = make_float2(ex2(x.x), ex2(x.y));
                const float vs = lo_f(vsm[j]), mid = fmaf(vs, 8.f, hi_f(vsm[j]));  // what code 8 stands for
                sum = __fadd2_rn(sum, p);
                low = __ffma2_rn(p, make_float2(mid, mid), low);
                const float2 y = __fmul2_rn(p, make_float2(vs, vs));
                P[j] = transposed(pack2(y.x, y.y));
            }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    l[e] *= al[e];
                    vmin[0][e] *= al[e];
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        O[0][w][e] *= al[e];
                        O[0][w][2 + e] *= al[e];
                    }
                }
            }
            l[0] += sum.x;
            l[1] += sum.y;
            vmin[0][0] += low.x;
            vmin[0][1] += low.y;
            // O^T += V^T P^T, 16 keys at a time
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t vf[2][8];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t A = *reinterpret_cast<const uint32_t*>(sv + 32 * (16 * i + 8 * x) + off_a);
                    const uint32_t B = *reinterpret_cast<const uint32_t*>(sv + 32 * (16 * i + 8 * x) + off_b);
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const uint32_t y = __byte_perm(A, B, w | (w << 4) | ((4 + w) << 8) | ((4 + w) << 12));
                        vf[x][2 * w] = centred((y & 0x000f000fu) | 0x43004300u);
                        vf[x][2 * w + 1] = centred(((y >> 4) & 0x000f000fu) | 0x43004300u);
                    }
                }
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const uint32_t A[4] = {vf[0][2 * w], vf[0][2 * w + 1], vf[1][2 * w], vf[1][2 * w + 1]};
                    mma16816(O[0][w], A, P[2 * i], P[2 * i + 1]);
                }
            }
        } else if constexpr (C::MMA) {
            float S[MT][4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                uint32_t kf[8];
                if constexpr (F == F_BF16) {
                    const uint4 x = *reinterpret_cast<const uint4*>(sk + 1024 * j + off_k);
                    const uint4 y = *reinterpret_cast<const uint4*>(sk + 1024 * j + (off_k ^ 64));
                    kf[0] = x.x, kf[1] = x.y, kf[2] = x.z, kf[3] = x.w, kf[4] = y.x, kf[5] = y.y, kf[6] = y.z, kf[7] = y.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2*>(sk + 256 * j + off_k);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        kf[i] = ((x.x >> (4 * i)) & 0x000f000fu) | 0x43004300u;
                        kf[4 + i] = ((x.y >> (4 * i)) & 0x000f000fu) | 0x43004300u;
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        if (ks == 0)
                            mma16816_0(S[mt][j], qf[mt][ks], kf[2 * ks], kf[2 * ks + 1]);
                        else
                            mma16816(S[mt][j], qf[mt][ks], kf[2 * ks], kf[2 * ks + 1]);
                    }
                }
            }
            uint32_t ksm[4][2], vsm[4][2];
            if constexpr (C::I4) {
                const uint32_t* ps = reinterpret_cast<const uint32_t*>(sk + C::SMO);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    ksm[j][0] = ps[8 * j + ka];
                    ksm[j][1] = ps[8 * j + kb];
                    vsm[j][0] = ps[KS + 8 * j + ka];
                    vsm[j][1] = ps[KS + 8 * j + kb];
                }
            }
            if constexpr (C::I4) {
                if (!whole) {  // scales of keys that are not there may be anything
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int k = 8 * j + (e ? kb : ka);
                            if (!((keep >> k) & 1)) ksm[j][e] = vsm[j][e] = 0;
                            if (alone >> k & 1) {  // (scale or least value is not finite: no dim of the row is)
                                vsm[j][e] = 0;
#pragma unroll
                                for (int r = 0; r < 2 * MT; ++r)
                                    if (sees(a, pos[r], base + k)) vmin[r >> 1][r & 1] = NAN;
                            }
                        }
                }
            }
            // scale and least value of a key's row enter its score, the codes' offset of 128 leaves:
            // q . k = scale * (q . (c + 128)) + (least - 128 scale) * sum q   (two columns at once)
            if constexpr (C::I4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 sc = make_float2(lo_f(ksm[j][0]), lo_f(ksm[j][1]));
                    const float2 off = __ffma2_rn(sc, make_float2(-128.f, -128.f), make_float2(hi_f(ksm[j][0]), hi_f(ksm[j][1])));
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int u = 0; u < 2; ++u) {
                            const float qs = qsum[mt][u];
                            const float2 y = __ffma2_rn(make_float2(S[mt][j][2 * u], S[mt][j][2 * u + 1]), sc,
                                                        __fmul2_rn(off, make_float2(qs, qs)));
                            S[mt][j][2 * u] = y.x;
                            S[mt][j][2 * u + 1] = y.y;
                        }
                }
            }
            if (!whole) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int k = 8 * j + ((x & 1) ? kb : ka);
                            if (!((keep >> k) & 1) || !sees(a, pos[2 * mt + (x >> 1)], base + k)) S[mt][j][x] = -INFINITY;
                        }
            }
            float2 vsc[4], mid[4];  // the values' scales, and what code 8 stands for
            if constexpr (C::I4) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    vsc[j] = make_float2(lo_f(vsm[j][0]), lo_f(vsm[j][1]));
                    mid[j] = __ffma2_rn(vsc[j], make_float2(8.f, 8.f), make_float2(hi_f(vsm[j][0]), hi_f(vsm[j][1])));
                }
            }
            uint32_t P[MT][4][2];  // [tile][rows g, g + 8]: the pair of columns
            bool grow = false;
            float al[2 * MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int j = 0; j < 4; ++j) mx = tc::fmax3(mx, S[mt][j][2 * u], S[mt][j][2 * u + 1]);
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * a.scale_log2;
                    // the maximum follows only when it grows by more than 2^8 (fp32 sums absorb that)
                    float& mm = m[2 * mt + u];
                    al[2 * mt + u] = 1.f;
                    if (mx > mm + 8.f || (mm == -INFINITY && mx > mm)) {
                        al[2 * mt + u] = ex2(mm - mx);
                        mm = mx;
                        grow = true;
                    }
                    const float mz = mm == -INFINITY ? 0.f : mm;
                    const float2 sc2 = make_float2(a.scale_log2, a.scale_log2), mz2 = make_float2(-mz, -mz);
                    float2 sum = make_float2(0.f, 0.f), low = make_float2(0.f, 0.f);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 x = __ffma2_rn(make_float2(S[mt][j][2 * u], S[mt][j][2 * u + 1]), sc2, mz2);
                        float2 p = make_float2(ex2(x.x), ex2(x.y));
                        sum = __fadd2_rn(sum, p);
                        if constexpr (C::I4) {
                            low = __ffma2_rn(p, mid[j], low);
                            p = __fmul2_rn(p, vsc[j]);
                        }
                        P[mt][j][u] = pack2(p.x, p.y);
                    }
                    l[2 * mt + u] = fmaf(l[2 * mt + u], al[2 * mt + u], sum.x + sum.y);
                    if constexpr (C::I4) vmin[mt][u] = fmaf(vmin[mt][u], al[2 * mt + u], low.x + low.y);
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
#pragma unroll
                        for (int nt = 0; nt < 8; ++nt) O[mt][nt][x] *= al[2 * mt + (x >> 1)];
                    }
            }
            // O += P V, 16 keys at a time: keys (tk(2c), tk(2c+1)) of tiles 2 i and 2 i + 1
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t vf[2][8];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int ta = 16 * i + 8 * x + ka, tb = 16 * i + 8 * x + kb;
                    if constexpr (F == F_BF16) {
                        const uint4 A = *reinterpret_cast<const uint4*>(sv + 128 * (16 * i + 8 * x) + off_a);
                        const uint4 B = *reinterpret_cast<const uint4*>(sv + 128 * (16 * i + 8 * x) + off_b);
                        const uint32_t av[4] = {A.x, A.y, A.z, A.w}, bv[4] = {B.x, B.y, B.z, B.w};
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            vf[x][2 * w] = __byte_perm(av[w], bv[w], 0x5410);
                            vf[x][2 * w + 1] = __byte_perm(av[w], bv[w], 0x7632);
                        }
                        if (!whole) {  // 0 x NaN is NaN: rows that are not there become zeros
                            const uint32_t in = keep & ~alone, z = (((in >> ta) & 1) ? 0xffffu : 0u) | (((in >> tb) & 1) ? 0xffff0000u : 0u);
#pragma unroll
                            for (int w = 0; w < 8; ++w) vf[x][w] &= z;
                        }
                    } else {
                        const uint32_t A = *reinterpret_cast<const uint32_t*>(sv + 32 * (16 * i + 8 * x) + off_a);
                        const uint32_t B = *reinterpret_cast<const uint32_t*>(sv + 32 * (16 * i + 8 * x) + off_b);
#pragma unroll
                        for (int w = 0; w < 4; ++w) {
                            const uint32_t y = __byte_perm(A, B, w | (w << 4) | ((4 + w) << 8) | ((4 + w) << 12));
                            vf[x][2 * w] = centred((y & 0x000f000fu) | 0x43004300u);
                            vf[x][2 * w + 1] = centred(((y >> 4) & 0x000f000fu) | 0x43004300u);
                        }
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const uint32_t pa[4] = {P[mt][2 * i][0], P[mt][2 * i][1], P[mt][2 * i + 1][0], P[mt][2 * i + 1][1]};
#pragma unroll
                    for (int nt = 0; nt < 8; ++nt) mma16816(O[mt][nt], pa, vf[0][nt], vf[1][nt]);
                }
            }
            if constexpr (!C::I4) {
                if (alone) {  // rare
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll 1
                        for (uint32_t left = (alone >> (8 * j)) & 0xff; left; left &= left - 1) {
                            // the key's column of P is with lane `from` of the row's four, dims 16 c .. with this one
                            const int x = __ffs(left) - 1, k = 8 * j + x, from = (lane & ~3) | (x < 4 ? x : (x + 2) & 3);
                            float p[MT][2];
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                for (int u = 0; u < 2; ++u) {
                                    const uint32_t w = __shfl_sync(0xffffffffu, P[mt][j][u], from);
                                    p[mt][u] = x < 4 ? lo_f(w) : hi_f(w);
                                }
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint4 y = *reinterpret_cast<const uint4*>(sv + 128 * k + (((2 * c + e) ^ (k & 7)) << 4));
                                const uint32_t v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                    for (int u = 0; u < 2; ++u) {
                                        if (!sees(a, pos[2 * mt + u], base + k)) continue;
#pragma unroll
                                        for (int z = 0; z < 4; ++z) {
                                            O[mt][2 * z][2 * u + e] = fmaf(p[mt][u], lo_f(v[z]), O[mt][2 * z][2 * u + e]);
                                            O[mt][2 * z + 1][2 * u + e] = fmaf(p[mt][u], hi_f(v[z]), O[mt][2 * z + 1][2 * u + e]);
                                        }
                                    }
                            }
                        }
                }
            }
        } else {
            // fp32: lane = key for the scores
            float* const pw = reinterpret_cast<float*>(sq + C::ROWS * 256);
            float kx[D];
            if constexpr (!C::I4) {
#pragma unroll
                for (int x = 0; x < 16; ++x)
                    *reinterpret_cast<float4*>(kx + 4 * x) = *reinterpret_cast<const float4*>(sk + (x >> 3) * KS * 128 + lane * 128 + (((x & 7) ^ (lane & 7)) << 4));
            } else {
                const uint32_t sm = *reinterpret_cast<const uint32_t*>(sk + C::SMO + lane * 4);
#pragma unroll
                for (int w = 0; w < 8; ++w) {
                    const uint32_t u = *reinterpret_cast<const uint32_t*>(sk + lane * 32 + w * 4);
#pragma unroll
                    for (int x = 0; x < 8; ++x) kx[8 * w + x] = fmaf(lo_f(sm), (float)((u >> (4 * x)) & 15), hi_f(sm));
                }
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                if (r >= nr) break;
                const float* q = reinterpret_cast<const float*>(sq) + r * D;
                float2 s0 = make_float2(0.f, 0.f), s1 = s0;  // (short chains: few warps hide little)
#pragma unroll
                for (int x = 0; x < D; x += 4) {
                    const float4 y = *reinterpret_cast<const float4*>(q + x);
                    s0 = __ffma2_rn(make_float2(y.x, y.y), make_float2(kx[x], kx[x + 1]), s0);
                    s1 = __ffma2_rn(make_float2(y.z, y.w), make_float2(kx[x + 2], kx[x + 3]), s1);
                }
                float s = (s0.x + s0.y) + (s1.x + s1.y);
                s = whole || (((keep >> lane) & 1) && sees(a, oldest + r0 + r - ap.by_t.div(r0 + r) * a.T, base + lane)) ? s * a.scale_log2 : -INFINITY;
                const float mn = fmaxf(m[r], warp_max(s));
                const float mz = mn == -INFINITY ? 0.f : mn;
                const float al = exp2f(m[r] - mz), p = exp2f(s - mz);
                m[r] = mn;
                l[r] = l[r] * al + p;  // (this lane's keys)
                acc[r][0] *= al;
                acc[r][1] *= al;
                pw[r * KS + lane] = p;
            }
            __syncwarp();
            // two dims a lane for the sum, four keys at once
            auto value = [&](int t) {
                if constexpr (!C::I4) {
                    return *reinterpret_cast<const float2*>(sv + (lane >> 4) * KS * 128 + t * 128 + ((((lane >> 1) & 7) ^ (t & 7)) << 4) + (lane & 1) * 8);
                } else {
                    const uint32_t sm = *reinterpret_cast<const uint32_t*>(sk + C::SMO + KS * 4 + t * 4);
                    const uint32_t u = sv[t * 32 + lane];
                    return make_float2(fmaf(lo_f(sm), (float)(u & 15), hi_f(sm)), fmaf(lo_f(sm), (float)(u >> 4), hi_f(sm)));
                }
            };
            const uint32_t with = keep & ~alone;
#pragma unroll 2
            for (int t = 0; t < KS; t += 4) {
                float2 v[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    v[x] = value(t + x);
                    if (!((with >> (t + x)) & 1)) v[x] = make_float2(0.f, 0.f);  // (0 x NaN is NaN)
                }
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    if (r >= nr) break;
                    const float4 p = *reinterpret_cast<const float4*>(pw + r * KS + t);
                    float2 y = make_float2(acc[r][0], acc[r][1]);
                    y = __ffma2_rn(make_float2(p.x, p.x), v[0], y);
                    y = __ffma2_rn(make_float2(p.y, p.y), v[1], y);
                    y = __ffma2_rn(make_float2(p.z, p.z), v[2], y);
                    y = __ffma2_rn(make_float2(p.w, p.w), v[3], y);
                    acc[r][0] = y.x;
                    acc[r][1] = y.y;
                }
            }
#pragma unroll 1
            for (uint32_t left = alone; left; left &= left - 1) {  // rare
                const int t = __ffs(left) - 1;
                const float2 v = value(t);
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    if (r >= nr) break;
                    if (!sees(a, oldest + r0 + r - ap.by_t.div(r0 + r) * a.T, base + t)) continue;
                    const float w = pw[r * KS + t];
                    acc[r][0] = fmaf(w, v.x, acc[r][0]);
                    acc[r][1] = fmaf(w, v.y, acc[r][1]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(empty(ring_id, st));  // the stage may be filled again
        if (++st == C::STAGES) st = 0, phase ^= 1;

        // the end of the item, or of this warp's part
        const bool last = cp.step + 1 == cp.s.steps;
        if (last || at + 1 == count) {
            const bool direct = last && at - seg + 1 == cp.s.steps;
            float* const part = a.part + (size_t)(2 * gw + (seg == 0 ? 0 : 1)) * ap.pl.slot;
            if constexpr (C::SWAP) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = 2 * c + e;
                    float ls = l[e], add = vmin[0][e];
#pragma unroll
                    for (int o = 4; o < 32; o <<= 1) {
                        ls += __shfl_xor_sync(0xffffffffu, ls, o);
                        add += __shfl_xor_sync(0xffffffffu, add, o);
                    }
                    if (r >= nr) continue;
                    const float mul = direct ? (ls > 0.f ? 1.f / ls : 0.f) : 1.f;
                    float y[8];
#pragma unroll
                    for (int w = 0; w < 8; ++w) y[w] = (O[0][w >> 1][2 * (w & 1) + e] + add) * mul;
                    if (direct) {
                        const int gt = r0 + r;
                        __nv_bfloat16* o = a.out.at<__nv_bfloat16>(cp.b, hk * a.G + gt / a.T, gt % a.T) + 8 * g;
                        *reinterpret_cast<uint4*>(o) = make_uint4(pack2(y[0], y[1]), pack2(y[2], y[3]), pack2(y[4], y[5]), pack2(y[6], y[7]));
                    } else {
                        float* o = part + (size_t)r * (D + 2);
#pragma unroll
                        for (int w = 0; w < 8; w += 2) *reinterpret_cast<float2*>(o + 8 * g + w) = make_float2(y[w], y[w + 1]);
                        if (g == 0) *reinterpret_cast<float2*>(o + D) = make_float2(m[e], ls);
                    }
                }
            } else if constexpr (C::MMA) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const int r = mt * 16 + g + 8 * u;
                        float ls = l[2 * mt + u], add = C::I4 ? vmin[mt][u] : 0.f;
                        ls += __shfl_xor_sync(0xffffffffu, ls, 1);
                        ls += __shfl_xor_sync(0xffffffffu, ls, 2);
                        if constexpr (C::I4) {
                            add += __shfl_xor_sync(0xffffffffu, add, 1);
                            add += __shfl_xor_sync(0xffffffffu, add, 2);
                        }
                        if (r >= nr) continue;
                        const float mul = direct ? (ls > 0.f ? 1.f / ls : 0.f) : 1.f;
                        float y[16];
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int nt = 0; nt < 8; ++nt) y[8 * e + nt] = (O[mt][nt][2 * u + e] + add) * mul;
                        if (direct) {
                            const int gt = r0 + r;
                            __nv_bfloat16* o = a.out.at<__nv_bfloat16>(cp.b, hk * a.G + gt / a.T, gt % a.T) + 16 * c;
#pragma unroll
                            for (int x = 0; x < 2; ++x)
                                reinterpret_cast<uint4*>(o)[x] =
                                    make_uint4(pack2(y[8 * x], y[8 * x + 1]), pack2(y[8 * x + 2], y[8 * x + 3]),
                                               pack2(y[8 * x + 4], y[8 * x + 5]), pack2(y[8 * x + 6], y[8 * x + 7]));
                        } else {
                            float* o = part + (size_t)r * (D + 2);
#pragma unroll
                            for (int x = 0; x < 16; x += 2) *reinterpret_cast<float2*>(o + 16 * c + x) = make_float2(y[x], y[x + 1]);
                            if (c == 0) *reinterpret_cast<float2*>(o + D) = make_float2(m[2 * mt + u], ls);
                        }
                    }
            } else {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    if (r >= nr) break;
                    const float ls = warp_sum(l[r]);
                    if (direct) {
                        const float mul = ls > 0.f ? 1.f / ls : 0.f;
                        const int gt = r0 + r;
                        float* o = a.out.at<float>(cp.b, hk * a.G + gt / a.T, gt % a.T) + 2 * lane;
                        o[0] = acc[r][0] * mul;
                        o[1] = acc[r][1] * mul;
                    } else {
                        float* o = part + (size_t)r * (D + 2);
                        *reinterpret_cast<float2*>(o + 2 * lane) = make_float2(acc[r][0], acc[r][1]);
                        if (lane == 0) *reinterpret_cast<float2*>(o + D) = make_float2(m[r], ls);
                    }
                }
            }
            fresh = true;
        }
        cp.next(a, tiles, false);
    }
}

// Parts of an item joined, JW warps a query row, in a fixed order: warp x takes every
// JW-th part of the warps that made them, eight loads under way at once, then the JW sums
// are added up in turn.  Sixteen warps where items are few and so have many parts, one
// where they are many (a block then takes sixteen rows).
constexpr int JT = 512;
template <typename T, int JW> __global__ void __launch_bounds__(JT) paged_join_kernel(const __grid_constant__ AttnP ap) {
    __shared__ float sums[JT / 32][D + 2];
    const PagedArgs& a = ap.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, jw = JW == 1 ? 0 : warp;
    const int w = JW == 1 ? (int)blockIdx.x * (JT / 32) + warp : (int)blockIdx.x;
    if (JW == 1 && w >= a.B * a.Hkv * ap.R) return;
    const int bk = w / ap.R, gt = w - bk * ap.R, b = bk / a.Hkv, hk = bk - b * a.Hkv;
    const int tiles = ap.pl.tiles, items = a.Hkv * tiles, tile = gt / ap.pl.rows, r = gt - tile * ap.pl.rows;
    const int h = hk * a.G + ap.by_t.div(gt), t = gt - ap.by_t.div(gt) * a.T;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the parts are there
    const int before = ap.first[b], steps = ap.first[b + 1] - before;
    const Parts parts(ap.first[a.B] * items, ap.pl.warps);
    const int first = before * items + (hk * tiles + tile) * steps;
    const int w0 = parts.of(first), w1 = parts.of(first + steps - 1);
    if (w0 == w1) return;  // written by its warp
    const bool at_begin = parts.begin(w0) == first;
    auto part = [&](int x) { return a.part + (size_t)(2 * x + (x > w0 || at_begin ? 0 : 1)) * ap.pl.slot + (size_t)r * (D + 2); };
    float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f;
    for (int x0 = w0 + jw; x0 <= w1; x0 += 8 * JW) {
        float2 ml[8], o[8];
        float mn = m;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const int x = x0 + u * JW;
            ml[u] = make_float2(-INFINITY, 0.f);
            o[u] = make_float2(0.f, 0.f);
            if (x <= w1) {
                const float* p = part(x);
                ml[u] = *reinterpret_cast<const float2*>(p + D);
                o[u] = *reinterpret_cast<const float2*>(p + 2 * lane);
            }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) mn = fmaxf(mn, ml[u].x);
        const float mz = mn == -INFINITY ? 0.f : mn, f0 = exp2f(m - mz);
        l *= f0;
        o0 *= f0;
        o1 *= f0;
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float f = exp2f(ml[u].x - mz);
            l = fmaf(ml[u].y, f, l);
            o0 = fmaf(o[u].x, f, o0);
            o1 = fmaf(o[u].y, f, o1);
        }
        m = mn;
    }
    if (JW > 1) {
        *reinterpret_cast<float2*>(&sums[warp][2 * lane]) = make_float2(o0, o1);
        if (lane == 0) *reinterpret_cast<float2*>(&sums[warp][D]) = make_float2(m, l);
        __syncthreads();
        if (warp != 0) return;
#pragma unroll
        for (int x = 1; x < JW; ++x) m = fmaxf(m, sums[x][D]);
        const float mz = m == -INFINITY ? 0.f : m;
        l = o0 = o1 = 0.f;
#pragma unroll
        for (int x = 0; x < JW; ++x) {
            const float f = exp2f(sums[x][D] - mz);
            l = fmaf(sums[x][D + 1], f, l);
            o0 = fmaf(sums[x][2 * lane], f, o0);
            o1 = fmaf(sums[x][2 * lane + 1], f, o1);
        }
    }
    const float il = l > 0.f ? 1.f / l : 0.f;
    T* out = a.out.at<T>(b, h, t) + 2 * lane;
    out[0] = from_f<T>(o0 * il);
    out[1] = from_f<T>(o1 * il);
}

size_t first_bytes(const PagedArgs& a) { return ((size_t)(a.B + 1) * 4 + 255) / 256 * 256; }

template <int F, int MT> cudaError_t run(const PagedArgs& a, cudaStream_t s) {
    using C = Cfg<F, MT>;
    AttnP p;
    p.a = a;
    p.R = a.G * a.T;
    p.pl = plan_for<F, MT>(p.R);
    p.by_t = FastDiv((uint32_t)a.T);
    p.by_half = FastDiv((uint32_t)(a.r ? a.r / 2 : 1));
    p.first = reinterpret_cast<int*>(a.part);
    p.a.part = reinterpret_cast<float*>(reinterpret_cast<char*>(a.part) + first_bytes(a));
    p.run = a.page_size < KS ? a.page_size : KS;
    p.run_bits = a.page_size < KS ? a.page_bits : 5;
    p.all_runs = (1u << (KS / p.run)) - 1;
    CUtensorMap mk{}, mv{};
    if (F == F_BF16) {
        // rows of every page as one long list
        const uint64_t rows = (uint64_t)a.n_pages * a.Hkv * a.page_size;
        if (!make_tmap_bf16_4d(&mk, a.k, rows, 1, 1, D, 0, 0, p.run, 2) || !make_tmap_bf16_4d(&mv, a.v, rows, 1, 1, D, 0, 0, p.run, 2))
            return cudaErrorInvalidValue;
    }
    if (F == F_FP32) {
        const uint64_t rows = (uint64_t)a.n_pages * a.Hkv * a.page_size;
        if (!make_tmap_f32_rows(&mk, a.k, rows, p.run) || !make_tmap_f32_rows(&mv, a.v, rows, p.run)) return cudaErrorInvalidValue;
    }
    cudaError_t e = allow_smem<paged_attn_kernel<F, MT>>(C::SMEM);
    if (e != cudaSuccess) return e;
    paged_attn_kernel<F, MT><<<NSM, C::THREADS, C::SMEM, s>>>(mk, mv, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int64_t rows = (int64_t)a.B * a.Hkv * p.R;
    // launched beside the first kernel: it is ready when that one ends
    cudaLaunchConfig_t cfg{};
    const bool many = (int64_t)a.B * a.Hkv * p.pl.tiles * 4 >= p.pl.warps;  // (then about five parts an item)
    cfg.gridDim = dim3((unsigned)(many ? (rows + JT / 32 - 1) / (JT / 32) : rows));
    cfg.blockDim = dim3(JT);
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return many ? cudaLaunchKernelEx(&cfg, paged_join_kernel<typename C::T, 1>, p)
                : cudaLaunchKernelEx(&cfg, paged_join_kernel<typename C::T, JT / 32>, p);
}

// f<format, m-tiles>() for the call's format and row count: 32 rows at once from 17 on, and in 4
// bits up to 8 as the products' columns (m-tiles 0)
template <class Fn> auto dispatch(const PagedArgs& a, Fn&& f) {
    const bool wide = a.G * a.T > 16;
    if (a.bf16 && !a.int4) return wide ? f.template operator()<F_BF16, 2>() : f.template operator()<F_BF16, 1>();
    if (a.bf16 && a.G * a.T <= 8) return f.template operator()<F_I4, 0>();
    if (a.bf16) return wide ? f.template operator()<F_I4, 2>() : f.template operator()<F_I4, 1>();
    return a.int4 ? f.template operator()<F_I4_FP32, 1>() : f.template operator()<F_FP32, 1>();
}
struct ScratchOf {
    const PagedArgs& a;
    template <int F, int MT> size_t operator()() const {
        const Plan p = plan_for<F, MT>(a.G * a.T);
        return first_bytes(a) + (size_t)p.warps * 2 * p.slot * sizeof(float);
    }
};
struct RunOf {
    const PagedArgs& a;
    cudaStream_t s;
    template <int F, int MT> cudaError_t operator()() const { return run<F, MT>(a, s); }
};

}  // namespace

size_t paged_attention_scratch(const PagedArgs& a) { return dispatch(a, ScratchOf{a}); }
cudaError_t launch_paged_attention(const PagedArgs& a, cudaStream_t s) { return dispatch(a, RunOf{a, s}); }

}  // namespace kvm
