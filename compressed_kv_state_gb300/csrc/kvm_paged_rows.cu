// Rows into and out of the paged cache: append (rotation and, for the 4-bit
// format, quantisation on the way) and read back.
//
// A row x of 64 values at position p: keys turn by the table's angles,
//   y_i = x_i cos - x_{i+r/2} sin,  y_{i+r/2} = x_{i+r/2} cos + x_i sin   (i < r/2),
// each product and sum rounded by itself.  INT4: least = bf16(min y), scale =
// bf16((max y - min y) / 15), code = clamp(rint((y - least) / scale), 0, 15).
//
// Reading is bound by the rows that go in and out (6.2 TB/s in bf16), the 4-bit append by
// instructions (issue 75%).  The plain append of a prompt is at 45% of the memory's rate (98 us
// for 32 x 8 x 4,096 rows): a row's loads wait for its length, start and page index, one after
// the other.  Eight lanes a row, each with eight
// neighbouring dims (16 bytes of bf16, 32 of fp32): four rows a warp instruction,
// every access whole sectors.  The rotation's partner dims come from the lane that
// holds them when the halves are whole pieces (r a multiple of 16), else from memory
// again.  Reading, a group of lanes takes four neighbouring tokens of a head (all their
// loads under way at once; 28 to 24 us for 8 ragged prompts of 4,000 tokens in 4 bits);
// appending one, as its arithmetic then has the warps that hide its latencies (four: 85 us
// against 56).
#include "kvm_paged.cuh"

namespace kvm {
namespace {

constexpr uint32_t ALL = 0xffffffffu;

// reductions over the eight lanes of a row
__device__ __forceinline__ float row_min(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v = fminf(v, __shfl_xor_sync(ALL, v, o));
    return v;
}
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(ALL, v, o));
    return v;
}

template <typename T> __device__ __forceinline__ void load8(const T* p, float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
        const uint4 u = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    } else {
        const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
        x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
    }
}
template <typename T> __device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
    if constexpr (sizeof(T) == 2) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
        *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
        *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// dims 8 c .. of a key row (x; the row at src) turned at position pos
template <typename T>
__device__ __forceinline__ void turn8(const PagedArgs& a, const T* src, int64_t pos, int c, float (&x)[8]) {
    const int half = a.r / 2;
    if (half == 0) return;
    const float2* cs_row = a.rope + pos * half;
    if ((half & 7) == 0) {
        const int hc = half >> 3;  // pieces of a half
        float y[8];
        const int from = (threadIdx.x & 24) + (c < hc ? c + hc : c < 2 * hc ? c - hc : c);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = __shfl_sync(ALL, x[i], from);
        if (c >= 2 * hc) return;
        const float4* tab = reinterpret_cast<const float4*>(cs_row + 8 * (c < hc ? c : c - hc));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 t = tab[i];
            const float s0 = c < hc ? -t.y : t.y, s1 = c < hc ? -t.w : t.w;
            x[2 * i] = __fadd_rn(__fmul_rn(x[2 * i], t.x), __fmul_rn(y[2 * i], s0));
            x[2 * i + 1] = __fadd_rn(__fmul_rn(x[2 * i + 1], t.z), __fmul_rn(y[2 * i + 1], s1));
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = 8 * c + i;
        if (d >= a.r) continue;
        const int pd = d < half ? d + half : d - half;
        const float2 cs = cs_row[d < half ? d : pd];
        x[i] = __fadd_rn(__fmul_rn(x[i], cs.x), __fmul_rn(to_f<T>(src[pd]), d < half ? -cs.y : cs.y));
    }
}

__device__ __forceinline__ float fmin3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __noinline__ uint32_t codes_divided(float x0, float x1, float x2, float x3, float x4, float x5, float x6, float x7,
                                               float s, float m) {
    auto code = [&](float x) { return (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x, m), s)), 0.f), 15.f); };
    return code(x0) | code(x1) << 4 | code(x2) << 8 | code(x3) << 12 | code(x4) << 16 | code(x5) << 20 | code(x6) << 24 |
           code(x7) << 28;
}

// The eight codes of x: rint((x - m) / s) held to 0..15, four bits each.  Almost always
// from a product with the reciprocal, in multiply-adds: u = the quotient / 15 held to
// 0..1, 15 u + 1.5 2^23 rounds it to a whole number.  That product is within 15 times a
// few units of the last place of the quotient, so only a row with a value closer than
// 1e-5 to a border is divided in full.
__device__ __forceinline__ uint32_t codes_of(const float (&x)[8], float s, float m) {
    const float k = __frcp_rn(s) * (1.f / 15.f), whole = 12582912.f;
    const float2 minus_m = make_float2(-m, -m), fifteen = make_float2(15.f, 15.f), up = make_float2(whole, whole),
                 down = make_float2(-whole, -whole);
    float r[8], far = 0.f;
#pragma unroll
    for (int u = 0; u < 8; u += 2) {  // (two at once; the same roundings)
        const float2 d = __fadd2_rn(make_float2(x[u], x[u + 1]), minus_m);
        const float2 q = make_float2(__saturatef(d.x * k), __saturatef(d.y * k));
        const float2 w = __fadd2_rn(__ffma2_rn(q, fifteen, up), down);
        const float2 off = __ffma2_rn(q, fifteen, make_float2(-w.x, -w.y));  // distance from the whole number
        r[u] = w.x;
        r[u + 1] = w.y;
        far = fmax3(far, fabsf(off.x), fabsf(off.y));
    }
    if (far > 0.49999f || !(s > 1e-30f)) return codes_divided(x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7], s, m);
    // sums below 2^16, exact; adding 2^23 leaves their bits at the bottom
    const float lo = fmaf(fmaf(fmaf(r[3], 16.f, r[2]), 16.f, r[1]), 16.f, r[0]);
    const float hi = fmaf(fmaf(fmaf(r[7], 16.f, r[6]), 16.f, r[5]), 16.f, r[4]);
    return __byte_perm(__float_as_uint(lo + 8388608.f), __float_as_uint(hi + 8388608.f), 0x5410);
}

// the tokens [i, i + TOK) of key head hk of sequence b that a group of eight lanes takes
template <int TOK> __device__ __forceinline__ bool my_tokens(const PagedArgs& a, int& b, int& hk, int& i) {
    const int64_t w = (blockIdx.x * 256ll + threadIdx.x) >> 3;
    const bool in = w < (int64_t)a.B * a.Hkv * a.by_n.d;
    const int x = in ? (int)w : 0, u = a.by_n.div(x);
    i = (x - u * (int)a.by_n.d) * TOK;
    b = a.by_h.div(u);
    hk = u - b * a.Hkv;
    return in;
}

template <typename T, bool I4> __global__ void __launch_bounds__(256) paged_append_kernel(const PagedArgs a) {
    const int c = threadIdx.x & 7;
    int b, hk, i;
    const bool in = my_tokens<1>(a, b, hk, i);  // (lanes past the end stay: rows share a warp's shuffles)
    bool live = in && (!a.lens || i < a.lens[b]);
    int64_t pos = 0, row = -1;
    if (live) {
        pos = a.start[b] + (int64_t)i;
        row = pos >= 0 && pos < a.cap ? paged_row(a, b, hk, pos) : -1;
        if (row < 0) {
            live = false;
            pos = 0;
            if (a.status && c == 0) atomicOr(a.status, KVM_DEV_DATA);
        }
    }
    if (!__any_sync(ALL, live)) return;
    float k[8] = {}, v[8] = {};
    const T* ks = a.rk.at<const T>(b, hk, i);
    if (live) {
        load8(ks + 8 * c, k);
        load8(a.rv.at<const T>(b, hk, i) + 8 * c, v);
    }
    turn8(a, ks, pos, c, k);
    if constexpr (!I4) {
        if (!live) return;
        store8(reinterpret_cast<T*>(a.k) + row * D + 8 * c, k);
        store8(reinterpret_cast<T*>(a.v) + row * D + 8 * c, v);
    } else {
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            float(&x)[8] = kv ? v : k;
            float2 f2 = make_float2(0.f, 0.f);
#pragma unroll
            for (int y = 0; y < 8; y += 2) f2 = __ffma2_rn(make_float2(x[y], x[y + 1]), make_float2(0.f, 0.f), f2);
            const float fin = f2.x + f2.y;  // not a number when some value is not finite
            const float lo = row_min(fmin3(fmin3(x[0], x[1], x[2]), fmin3(x[3], x[4], x[5]), fminf(x[6], x[7])));
            const float hi = row_max(fmax3(fmax3(x[0], x[1], x[2]), fmax3(x[3], x[4], x[5]), fmaxf(x[6], x[7])));
            const uint32_t odd = __ballot_sync(ALL, !(fin == 0.f));
            __nv_bfloat16 sc = __float2bfloat16_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.f)), mn = __float2bfloat16_rn(lo);
            if ((odd >> (threadIdx.x & 24)) & 0xff) sc = mn = __ushort_as_bfloat16(0x7fff);  // the whole row reads as NaN
            const float s = __bfloat162float(sc), m = __bfloat162float(mn);
            const uint32_t word = s > 0.f ? codes_of(x, s, m) : 0;
            if (!live) continue;
            reinterpret_cast<uint32_t*>(kv ? a.v : a.k)[row * 8 + c] = word;
            if (c == 0) (kv ? a.v_sm : a.k_sm)[row] = (uint32_t)__bfloat16_as_ushort(sc) | ((uint32_t)__bfloat16_as_ushort(mn) << 16);
        }
    }
}

// a group of lanes takes TOK neighbouring tokens
template <typename T, bool I4, int TOK> __global__ void __launch_bounds__(256) paged_read_kernel(const PagedArgs a) {
    const int c = threadIdx.x & 7;
    int b, hk, i0;
    if (!my_tokens<TOK>(a, b, hk, i0)) return;
    const int end = (int)min(a.n_new, a.lens ? (int64_t)a.lens[b] : a.n_new);
    const int64_t pos0 = a.start[b] + (int64_t)i0;
    T* kd = a.rk.at<T>(b, hk, i0) + 8 * c;
    T* vd = a.rv.at<T>(b, hk, i0) + 8 * c;
    int64_t row[TOK];
#pragma unroll
    for (int u = 0; u < TOK; ++u) {
        const int64_t pos = pos0 + u;
        row[u] = -1;
        if (i0 + u < end) {
            if (pos >= 0 && pos < (int64_t)a.max_pages * a.page_size) row[u] = paged_row(a, b, hk, pos);
            if (row[u] < 0 && a.status && c == 0) atomicOr(a.status, KVM_DEV_DATA);
        }
    }
    if constexpr (!I4) {
#pragma unroll
        for (int u = 0; u < TOK; ++u) {
            if (i0 + u >= a.n_new) break;
            float x[8] = {}, y[8] = {};
            if (row[u] >= 0) {
                load8(reinterpret_cast<const T*>(a.k) + row[u] * D + 8 * c, x);
                load8(reinterpret_cast<const T*>(a.v) + row[u] * D + 8 * c, y);
            }
            store8(kd + u * a.rk.sn, x);
            store8(vd + u * a.rv.sn, y);
        }
    } else {
        uint32_t word[TOK][2], sm[TOK][2];
#pragma unroll
        for (int u = 0; u < TOK; ++u) {
            word[u][0] = word[u][1] = sm[u][0] = sm[u][1] = 0;
            if (row[u] < 0) continue;
            word[u][0] = reinterpret_cast<const uint32_t*>(a.k)[row[u] * 8 + c];
            word[u][1] = reinterpret_cast<const uint32_t*>(a.v)[row[u] * 8 + c];
            sm[u][0] = a.k_sm[row[u]];
            sm[u][1] = a.v_sm[row[u]];
        }
#pragma unroll
        for (int u = 0; u < TOK; ++u) {
            if (i0 + u >= a.n_new) break;
#pragma unroll
            for (int kv = 0; kv < 2; ++kv) {
                const float s = __uint_as_float(sm[u][kv] << 16), m = __uint_as_float(sm[u][kv] & 0xffff0000u);
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // 16 + code from the code's bits; scale * code has 12 bits, so the multiply-add
                    // rounds once, as least + scale * code does
                    const uint32_t w = e < 5 ? word[u][kv] << (19 - 4 * e) : word[u][kv] >> (4 * e - 19);
                    x[e] = fmaf(s, __uint_as_float((w & 0x780000u) | 0x41800000u) - 16.f, m);
                }
                store8(kv ? vd + u * a.rv.sn : kd + u * a.rk.sn, x);
            }
        }
    }
}

}  // namespace

namespace {
template <class K> cudaError_t launch_rows(K kernel, int tok, const PagedArgs& a, cudaStream_t s) {
    PagedArgs p = a;
    p.by_n = FastDiv((uint32_t)((a.n_new + tok - 1) / tok));
    p.by_h = FastDiv((uint32_t)a.Hkv);
    const int64_t groups = (int64_t)a.B * a.Hkv * p.by_n.d;
    kernel<<<(unsigned)((groups + 31) / 32), 256, 0, s>>>(p);
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_paged_append(const PagedArgs& a, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (a.bf16) return a.int4 ? launch_rows(paged_append_kernel<B, true>, 1, a, s) : launch_rows(paged_append_kernel<B, false>, 1, a, s);
    return a.int4 ? launch_rows(paged_append_kernel<float, true>, 1, a, s) : launch_rows(paged_append_kernel<float, false>, 1, a, s);
}
cudaError_t launch_paged_read(const PagedArgs& a, cudaStream_t s) {
    using B = __nv_bfloat16;
    if (a.n_new < 64) {
        if (a.bf16) return a.int4 ? launch_rows(paged_read_kernel<B, true, 1>, 1, a, s) : launch_rows(paged_read_kernel<B, false, 1>, 1, a, s);
        return a.int4 ? launch_rows(paged_read_kernel<float, true, 1>, 1, a, s) : launch_rows(paged_read_kernel<float, false, 1>, 1, a, s);
    }
    if (a.bf16) return a.int4 ? launch_rows(paged_read_kernel<B, true, 4>, 4, a, s) : launch_rows(paged_read_kernel<B, false, 4>, 4, a, s);
    return a.int4 ? launch_rows(paged_read_kernel<float, true, 4>, 4, a, s) : launch_rows(paged_read_kernel<float, false, 4>, 4, a, s);
}

}  // namespace kvm
