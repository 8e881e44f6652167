// groupnorm.cu — group norm over channels-last rows with an optional SiLU,
// forward and vector-Jacobian product (sm_103a).
//
//   x [N, S, C], groups of C/G consecutive channels:  μ, r = 1/√(var + eps)
//   over the S·C/G values of a group of a sample,
//   x̂ = (x − μ)·r,  z = x̂·w + b,  y = z  or  z·sigmoid(z)
// Backward, with dz = dy  or  dy·silu′(z), per sample and channel
//   A = Σ_s dz·x̂,  B = Σ_s dz:   grad_w = Σ_n A,  grad_b = Σ_n B
// and per group  m₂ = Σ_c w·A / M,  m₁ = Σ_c w·B / M  (M = S·C/G):
//   dx = r·(dz·w − m₁ − x̂·m₂)
// so the groups' sums come from the channels', which the parameter gradients
// need anyway, and no thread has to know where a group begins or ends until
// a tile's channel sums are in shared memory.
//
// A thread keeps one 16-byte vector of channels and walks the rows of a
// tile.  Statistics of a tile: sums of x and x² about the thread's first
// value, then means and squared deviations of threads, and of tiles, joined
// about their common mean (no subtraction of large sums).
#include <stdint.h>

#include <algorithm>

#include "wsf_block.h"
#include "wsf_device.cuh"
#include "wsf_internal.h"

namespace wsf {
namespace {

constexpr int NT = 256;

// V consecutive elements as they are loaded (16 bytes, or one element), and as
// binary32.
template <typename T, int V>
struct Held {
    Raw16 raw;
    __device__ __forceinline__ void load(const T* p) { raw = ld_keep(p); }
    __device__ __forceinline__ void widen(float (&f)[V]) const { Elt<T>::widen(raw, f); }
};
template <typename T>
struct Held<T, 1> {
    float raw;
    __device__ __forceinline__ void load(const T* p) { raw = Elt<T>::load1(p); }
    __device__ __forceinline__ void widen(float (&f)[1]) const { f[0] = raw; }
};
template <typename T, int V>
__device__ __forceinline__ void store_v(T* p, const float (&f)[V]) {
    if constexpr (V == 1)
        Elt<T>::store1(p, f[0]);
    else
        st_stream(p, Elt<T>::narrow(f));
}

// sigmoid(z): for binary32 storage by expf and a true division, for 16-bit
// storage by the hardware's exponential and reciprocal (a few 2⁻²², far
// below the 2⁻¹¹ half step of the outputs).
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    if constexpr (sizeof(T) == 4)
        return 1.0f / (1.0f + expf(-z));
    else
        return __fdividef(1.0f, 1.0f + __expf(-z));
}
template <typename T, bool Silu>
__device__ __forceinline__ float activate(float z) {
    if constexpr (!Silu) return z;
    return z * sigmoid<T>(z);
}
// dy·silu′(z)
template <typename T, bool Silu>
__device__ __forceinline__ float through(float dy, float z) {
    if constexpr (!Silu) return dy;
    const float q = sigmoid<T>(z);
    return dy * q * fmaf(z, 1.0f - q, 1.0f);
}

struct Shape {
    int64_t N, S, xn, xs, yn, ys, gn, gs;  // strides of x, of y or dx, of dy
    int C, G, Cg;
    int tiles;     // row tiles of a sample
    int64_t rows;  // rows of a tile
};

// Threads of a block over a tile: cv vectors a row, RL rows at a time.
struct Lanes {
    int cv, RL, c, r;
    __device__ __forceinline__ Lanes(int C, int V) {
        cv = C / V;
        RL = cv < NT ? NT / cv : 1;
        c = cv < NT ? (int)threadIdx.x % cv : (int)threadIdx.x;
        r = cv < NT ? (int)threadIdx.x / cv : 0;
    }
};

// A unit is a tile of a sample.
struct Unit {
    int64_t n, tile, s0;
    int rows;
    __device__ __forceinline__ Unit(const Shape& d, int64_t u) {
        n = u / d.tiles;
        tile = u - n * d.tiles;
        s0 = tile * d.rows;
        rows = (int)min(d.rows, d.S - s0);
    }
};

// Rows of a tile that row lane r holds: r, r + RL, ...
struct Rows {
    int base, extra;
    __device__ __forceinline__ Rows(int rows, int RL) { base = rows / RL, extra = rows - base * RL; }
    __device__ __forceinline__ int of(int r) const { return base + (r < extra); }
};

// Groups of V consecutive channels from ch on, without a division a channel.
template <int V>
__device__ __forceinline__ void groups_of(int ch, int Cg, int (&g)[V]) {
    g[0] = ch / Cg;
    int left = (g[0] + 1) * Cg - ch;
#pragma unroll
    for (int i = 1; i < V; i++) {
        left--;
        const bool next = left == 0;
        g[i] = g[i - 1] + next;
        left = next ? Cg : left;
    }
}

// ---------------------------------------------------------------------------
// Any S: two passes over x, the second of which finds it in L2 (the host
// takes the samples in chunks that fit; the second pass walks the tiles
// backwards, so that of a sample that does not fit the end is still there).
//
// First pass: mean and squared deviations of every group over a tile.  A
// thread sums about its first value; threads' means and deviations are joined
// about their common mean, first the row lanes of a channel (Q threads a
// channel where there are few), then a group's channels by a warp.
template <typename T, int V>
__global__ void __launch_bounds__(NT, 4) gn_stats_kernel(const T* x, const Shape d, float2* part) {
    constexpr int U = V == 1 ? 8 : 4;
    extern __shared__ float4 smem[];
    const Lanes t(d.C, V);
    float* sm = reinterpret_cast<float*>(smem);  // [RL][C] means
    float* sq = sm + (size_t)t.RL * d.C;         // [RL][C] squared deviations
    pdl_wait();
    const Unit un(d, blockIdx.x);
    const Rows rows(un.rows, t.RL);
    const T* base = x + un.n * d.xn + un.s0 * d.xs;
    if (t.r < t.RL) {
        const int cnt = rows.of(t.r);
        const float inv = cnt ? 1.0f / cnt : 0.f;
        const int64_t step = t.RL * d.xs;
        for (int c = t.c; c < t.cv; c += NT) {
            float k[V], a[V], b[V];
#pragma unroll
            for (int i = 0; i < V; i++) k[i] = a[i] = b[i] = 0.f;
            const T* p = base + (int64_t)t.r * d.xs + c * V;
            if (cnt) {
                Held<T, V> h;
                h.load(p);
                h.widen(k);
            }
            for (int j = 1; j < cnt; j += U) {
                Held<T, V> h[U];
#pragma unroll
                for (int u = 0; u < U; u++) {
                    if (j + u < cnt) p += step;
                    h[u].load(p);
                }
#pragma unroll
                for (int u = 0; u < U; u++) {
                    if (j + u < cnt) {
                        float f[V];
                        h[u].widen(f);
#pragma unroll
                        for (int i = 0; i < V; i++) {
                            const float q = f[i] - k[i];
                            a[i] += q;
                            b[i] = fmaf(q, q, b[i]);
                        }
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < V; i++) {
                const float m = a[i] * inv;
                sm[t.r * d.C + c * V + i] = k[i] + m;
                sq[t.r * d.C + c * V + i] = fmaxf(fmaf(-m, a[i], b[i]), 0.f);
            }
        }
    }
    __syncthreads();
    // row lanes part, part + Q, ... of a channel, into lane `part`
    const int Q = d.C < NT ? min(NT / d.C, t.RL) : 1;
    const int part0 = d.C < NT ? (int)threadIdx.x / d.C : 0;
    if (t.RL > 1 && part0 < Q) {
        for (int c = d.C < NT ? (int)threadIdx.x % d.C : (int)threadIdx.x; c < d.C; c += NT) {
            float s = 0.f;
            int n = 0;
            for (int r = part0; r < t.RL; r += Q) {
                s = fmaf((float)rows.of(r), sm[r * d.C + c], s);
                n += rows.of(r);
            }
            const float m = n ? s / n : 0.f;
            s = 0.f;
            for (int r = part0; r < t.RL; r += Q) {
                const float e = sm[r * d.C + c] - m;
                s += fmaf((float)rows.of(r) * e, e, sq[r * d.C + c]);
            }
            sm[part0 * d.C + c] = m;
            sq[part0 * d.C + c] = s;
        }
    }
    __syncthreads();
    const int lane = threadIdx.x & 31;
    const float inv = 1.0f / ((float)un.rows * d.Cg);
    for (int g = threadIdx.x >> 5; g < d.G; g += NT / 32) {
        float s = 0.f, mean = 0.f;
#pragma unroll
        for (int pass = 0; pass < 2; pass++) {
            s = 0.f;
            for (int q = 0; q < Q; q++) {
                int n = 0;  // rows of the part
                for (int r = q; r < t.RL; r += Q) n += rows.of(r);
                for (int c = lane; c < d.Cg; c += 32) {
                    const int at = q * d.C + g * d.Cg + c;
                    const float e = sm[at] - mean;
                    s += pass ? fmaf((float)n * e, e, sq[at]) : (float)n * e;
                }
            }
            s = group_sum<32>(s);
            if (pass == 0) mean = s * inv;
        }
        if (lane == 0) part[(int64_t)blockIdx.x * d.G + g] = make_float2(mean, s);
    }
    pdl_trigger();
}

// Second pass.  The block first joins its sample's tiles, a warp a group; the
// first tile's block writes the statistics out.
template <typename T, int V, bool Silu>
__global__ void __launch_bounds__(NT, 4) gn_apply_kernel(const T* x, T* y, const float* w,
                                                      const float* b, float eps, float* mean,
                                                      float* rstd, const float2* part,
                                                      const Shape d) {
    constexpr int U = V == 1 ? 8 : 4;
    extern __shared__ float4 smem[];
    float2* st = reinterpret_cast<float2*>(smem);  // [G] mean, 1/deviation
    const Lanes t(d.C, V);
    pdl_wait();
    const Unit un(d, (int64_t)gridDim.x - 1 - blockIdx.x);
    {
        const int lane = threadIdx.x & 31;
        for (int g = threadIdx.x >> 5; g < d.G; g += NT / 32) {
            const float2* p = part + un.n * d.tiles * d.G + g;
            float s = 0.f;
            for (int i = lane; i < d.tiles; i += 32)
                s = fmaf((float)min(d.rows, d.S - i * d.rows), p[(int64_t)i * d.G].x, s);
            const float m = group_sum<32>(s) / (float)d.S;
            s = 0.f;
            for (int i = lane; i < d.tiles; i += 32) {
                const float2 q = p[(int64_t)i * d.G];
                const float e = q.x - m;
                s += fmaf((float)min(d.rows, d.S - i * d.rows) * d.Cg * e, e, q.y);
            }
            s = group_sum<32>(s);
            if (lane == 0) {
                const float r = 1.0f / sqrtf(s / ((float)d.S * d.Cg) + eps);
                st[g] = make_float2(m, r);
                if (un.tile == 0) mean[un.n * d.G + g] = m, rstd[un.n * d.G + g] = r;
            }
        }
    }
    __syncthreads();
    if (t.r < t.RL) {
        const int64_t xstep = t.RL * d.xs, ystep = t.RL * d.ys;
        const int cnt = Rows(un.rows, t.RL).of(t.r);
        for (int c = t.c; c < t.cv; c += NT) {
            float mu[V], rw[V], sh[V];
            int g[V];
            groups_of<V>(c * V, d.Cg, g);
#pragma unroll
            for (int i = 0; i < V; i++) {
                const float2 q = st[g[i]];
                mu[i] = q.x;
                rw[i] = q.y * __ldg(w + c * V + i);
                sh[i] = __ldg(b + c * V + i);
            }
            const T* p = x + un.n * d.xn + (un.s0 + t.r) * d.xs + c * V;
            T* o = y + un.n * d.yn + (un.s0 + t.r) * d.ys + c * V;
            for (int j = 0; j < cnt; j += U) {
                Held<T, V> h[U];
#pragma unroll
                for (int u = 0; u < U; u++) {
                    h[u].load(p);
                    if (j + u < cnt - 1) p += xstep;
                }
#pragma unroll
                for (int u = 0; u < U; u++) {
                    if (j + u < cnt) {
                        float f[V];
                        h[u].widen(f);
#pragma unroll
                        for (int i = 0; i < V; i++)
                            f[i] = activate<T, Silu>(fmaf(f[i] - mu[i], rw[i], sh[i]));
                        store_v<T, V>(o, f);
                        o += ystep;
                    }
                }
            }
        }
    }
    pdl_trigger();
}

// ---------------------------------------------------------------------------
// Backward, first pass: a block walks units u0 .. u1 and writes each unit's
// groups' sums (m₂, m₁ shares) and, over all of them, the channels' sums.
template <typename T, int V, bool Silu>
__global__ void __launch_bounds__(NT, 3) gn_bwd_sums_kernel(const T* x, const T* dy, const float* w,
                                                         const float* b, const float* mean,
                                                         const float* rstd, const Shape d,
                                                         float2* part_g, float* part_a,
                                                         float* part_b) {
    constexpr int U = 2;
    extern __shared__ float4 smem[];
    const Lanes t(d.C, V);
    float* sa = reinterpret_cast<float*>(smem);  // [RL][C]
    float* sb = sa + (size_t)t.RL * d.C;         // [RL][C]
    float* ta = part_a + (int64_t)blockIdx.x * d.C;  // [C] the block's own row
    float* tb = part_b + (int64_t)blockIdx.x * d.C;
    pdl_wait();
    const int64_t units = d.N * d.tiles;
    const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
    const int Q = d.C < NT ? min(NT / d.C, t.RL) : 1;
    const int part0 = d.C < NT ? (int)threadIdx.x / d.C : 0;
    for (int64_t u = u0; u < u1; u++) {
        const Unit un(d, u);
        if (t.r < t.RL) {
            const int64_t xstep = t.RL * d.xs, gstep = t.RL * d.gs;
            const int cnt = Rows(un.rows, t.RL).of(t.r);
            for (int c = t.c; c < t.cv; c += NT) {
                float mu[V], rw[V], bc[V], A[V], B[V];
                int g[V];
                groups_of<V>(c * V, d.Cg, g);
#pragma unroll
                for (int i = 0; i < V; i++) {
                    mu[i] = mean[un.n * d.G + g[i]];
                    rw[i] = rstd[un.n * d.G + g[i]] * __ldg(w + c * V + i);
                    bc[i] = __ldg(b + c * V + i);
                    A[i] = B[i] = 0.f;
                }
                const T* p = x + un.n * d.xn + (un.s0 + t.r) * d.xs + c * V;
                const T* q = dy + un.n * d.gn + (un.s0 + t.r) * d.gs + c * V;
                for (int j = 0; j < cnt; j += U) {
                    Held<T, V> hx[U], hg[U];
#pragma unroll
                    for (int k = 0; k < U; k++) {
                        hx[k].load(p);
                        hg[k].load(q);
                        if (j + k < cnt - 1) p += xstep, q += gstep;
                    }
#pragma unroll
                    for (int k = 0; k < U; k++) {
                        if (j + k < cnt) {
                            float f[V], h[V];
                            hx[k].widen(f);
                            hg[k].widen(h);
#pragma unroll
                            for (int i = 0; i < V; i++) {
                                f[i] -= mu[i];
                                const float dz = through<T, Silu>(h[i], fmaf(f[i], rw[i], bc[i]));
                                A[i] = fmaf(dz, f[i], A[i]);  // times r below
                                B[i] += dz;
                            }
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < V; i++) {
                    sa[t.r * d.C + c * V + i] = A[i] * rstd[un.n * d.G + g[i]];
                    sb[t.r * d.C + c * V + i] = B[i];
                }
            }
        }
        __syncthreads();
        if (t.RL > 1 && Q > 1 && part0 < Q) {  // row lanes of a channel, Q threads a channel
            const int c = (int)threadIdx.x % d.C;
            float A = 0.f, B = 0.f;
            for (int r = part0; r < t.RL; r += Q) A += sa[r * d.C + c], B += sb[r * d.C + c];
            sa[part0 * d.C + c] = A;
            sb[part0 * d.C + c] = B;
        }
        __syncthreads();
        const int left = Q > 1 ? Q : t.RL;
        for (int c = threadIdx.x; c < d.C; c += NT) {
            float A = sa[c], B = sb[c];
            for (int r = 1; r < left; r++) A += sa[r * d.C + c], B += sb[r * d.C + c];
            ta[c] = u > u0 ? ta[c] + A : A;
            tb[c] = u > u0 ? tb[c] + B : B;
            sa[c] = A * __ldg(w + c);
            sb[c] = B * __ldg(w + c);
        }
        __syncthreads();
        const int lane = threadIdx.x & 31;
        for (int g = threadIdx.x >> 5; g < d.G; g += NT / 32) {
            float A = 0.f, B = 0.f;
            for (int c = lane; c < d.Cg; c += 32) A += sa[g * d.Cg + c], B += sb[g * d.Cg + c];
            A = group_sum<32>(A);
            B = group_sum<32>(B);
            if (lane == 0) part_g[u * d.G + g] = make_float2(A, B);
        }
        __syncthreads();
    }
    pdl_trigger();
}

template <typename T, int V, bool Silu>
__global__ void __launch_bounds__(NT, 3) gn_bwd_apply_kernel(const T* x, const T* dy, T* dx,
                                                          const float* w, const float* b,
                                                          const float* mean, const float* rstd,
                                                          const float2* part, const Shape d) {
    constexpr int U = 2;
    extern __shared__ float4 smem[];
    float4* st = smem;  // [G] μ, r, r·m₁, r²·m₂
    const Lanes t(d.C, V);
    pdl_wait();
    const Unit un(d, (int64_t)gridDim.x - 1 - blockIdx.x);
    {
        const int lane = threadIdx.x & 31;
        const float inv = 1.0f / ((float)d.S * d.Cg);
        for (int g = threadIdx.x >> 5; g < d.G; g += NT / 32) {
            const float2* p = part + un.n * d.tiles * d.G + g;
            float A = 0.f, B = 0.f;
            for (int i = lane; i < d.tiles; i += 32) {
                const float2 q = p[(int64_t)i * d.G];
                A += q.x;
                B += q.y;
            }
            A = group_sum<32>(A);
            B = group_sum<32>(B);
            if (lane == 0) {
                const float r = rstd[un.n * d.G + g];
                st[g] = make_float4(mean[un.n * d.G + g], r, r * (B * inv), r * r * (A * inv));
            }
        }
    }
    __syncthreads();
    if (t.r < t.RL) {
        const int64_t xstep = t.RL * d.xs, gstep = t.RL * d.gs, ystep = t.RL * d.ys;
        const int cnt = Rows(un.rows, t.RL).of(t.r);
        for (int c = t.c; c < t.cv; c += NT) {
            // dx = dz·(w·r) − (x − μ)·(r²·m₂) − r·m₁
            float mu[V], rw[V], bc[V], e2[V], e1[V];
            int g[V];
            groups_of<V>(c * V, d.Cg, g);
#pragma unroll
            for (int i = 0; i < V; i++) {
                const float4 q = st[g[i]];
                mu[i] = q.x;
                rw[i] = q.y * __ldg(w + c * V + i);
                bc[i] = __ldg(b + c * V + i);
                e1[i] = q.z;
                e2[i] = q.w;
            }
            const T* p = x + un.n * d.xn + (un.s0 + t.r) * d.xs + c * V;
            const T* q = dy + un.n * d.gn + (un.s0 + t.r) * d.gs + c * V;
            T* o = dx + un.n * d.yn + (un.s0 + t.r) * d.ys + c * V;
            for (int j = 0; j < cnt; j += U) {
                Held<T, V> hx[U], hg[U];
#pragma unroll
                for (int k = 0; k < U; k++) {
                    hx[k].load(p);
                    hg[k].load(q);
                    if (j + k < cnt - 1) p += xstep, q += gstep;
                }
#pragma unroll
                for (int k = 0; k < U; k++) {
                    if (j + k < cnt) {
                        float f[V], h[V];
                        hx[k].widen(f);
                        hg[k].widen(h);
#pragma unroll
                        for (int i = 0; i < V; i++) {
                            f[i] -= mu[i];
                            const float dz = through<T, Silu>(h[i], fmaf(f[i], rw[i], bc[i]));
                            f[i] = fmaf(dz, rw[i], -fmaf(f[i], e2[i], e1[i]));
                        }
                        store_v<T, V>(o, f);
                        o += ystep;
                    }
                }
            }
        }
    }
    pdl_trigger();
}

// grad[c] (+)= Σ_p part[p, c] for both gradients: 32 columns by 32 stripes of
// rows (p ≡ stripe mod 32, in order), stripes joined by a fixed tree, in
// compensated pairs.
__global__ void __launch_bounds__(1024) gn_grad_kernel(const float* part_a, const float* part_b,
                                                       int64_t P, int C, float* gw, float* gb,
                                                       int accumulate) {
    __shared__ float2 st[32][33];
    pdl_wait();
    const int col = threadIdx.x & 31, stripe = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + col;
    const float* part = blockIdx.y ? part_b : part_a;
    float* out = blockIdx.y ? gb : gw;
    Acc2 a = acc2_zero();
    if (c < C)
        for (int64_t p = stripe; p < P; p += 32) acc2_add1(a, part[p * C + c]);
    st[stripe][col] = make_float2(a.hi, a.lo);
    __syncthreads();
    for (int h = 16; h > 0; h >>= 1) {
        if (stripe < h) {
            const float2 o = st[stripe + h][col];
            a = acc2_add(a, Acc2{o.x, o.y});
            st[stripe][col] = make_float2(a.hi, a.lo);
        }
        __syncthreads();
    }
    if (stripe == 0 && c < C) {
        const float v = acc2_value(a);
        out[c] = accumulate ? out[c] + v : v;
    }
    pdl_trigger();
}

// ---------------------------------------------------------------------------
// Rows of heads (S == 1): a group is one contiguous run that lpg lanes hold,
// CPL 16-byte vectors a lane, so both statistics, and the backward's two
// group sums, are butterflies over those lanes and every value is read once.
// A warp keeps its place in the row (w, b and the gradient sums stay in
// registers) and walks the samples, U of them in flight.
constexpr int RT = 256, RW = RT / 32;

struct RowShape {
    int64_t N, xn, yn, gn;
    int C, G, Cg;
    int lpg, cpg;   // lanes of a group (a power of two), vectors of a group
    int spr, rpw;   // lanes of a row, rows of a warp (1 if a row fills it)
    int segs, RB;   // grid: warps that a row spreads over, blocks along the samples
};

// A lane's place: its group, its vectors' first element, its row of the warp.
struct Place {
    int g, j, sub, at;
    bool on;
    __device__ __forceinline__ Place(const RowShape& d, int V) {
        const int lane = threadIdx.x & 31, seg = blockIdx.x % d.segs;
        const int slot = d.rpw > 1 ? lane % d.spr : seg * 32 + lane;
        sub = d.rpw > 1 ? lane / d.spr : 0;
        on = slot < d.spr && sub < d.rpw;
        g = on ? slot / d.lpg : 0;
        j = slot & (d.lpg - 1);
        at = g * d.Cg + j * V;
    }
};

__device__ __forceinline__ float lanes_sum(float v, int lpg) {
    for (int o = lpg >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    return v;
}

template <typename T, int CPL, bool Silu>
__global__ void __launch_bounds__(RT, CPL == 1 ? 3 : 2)
    gn_rows_fwd_kernel(const T* x, T* y, const float* w, const float* b, float eps, float* mean,
                       float* rstd, const RowShape d) {
    constexpr int V = Elt<T>::V, U = CPL == 1 ? 4 : 2;
    const Place t(d, V);
    const float inv = 1.0f / (float)d.Cg;
    bool has[CPL];
    float wc[CPL][V], bc[CPL][V];
    pdl_wait();
#pragma unroll
    for (int c = 0; c < CPL; c++) {
        has[c] = t.on && t.j + c * d.lpg < d.cpg;
#pragma unroll
        for (int i = 0; i < V; i++) {
            wc[c][i] = has[c] ? __ldg(w + t.at + c * d.lpg * V + i) : 0.f;
            bc[c][i] = has[c] ? __ldg(b + t.at + c * d.lpg * V + i) : 0.f;
        }
    }
    const int64_t step = (int64_t)d.RB * RW * d.rpw;
    const int64_t first = ((int64_t)(blockIdx.x / d.segs) * RW + (threadIdx.x >> 5)) * d.rpw;
    for (int64_t n0 = first; n0 < d.N; n0 += U * step) {
        Raw16 raw[U][CPL];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int64_t n = n0 + u * step + t.sub;
#pragma unroll
            for (int c = 0; c < CPL; c++)
                raw[u][c] = has[c] && n < d.N ? ld_stream(x + n * d.xn + t.at + c * d.lpg * V)
                                              : raw_zero();
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (n0 + u * step >= d.N) break;
            const int64_t n = n0 + u * step + t.sub;
            float f[CPL][V], s = 0.f;
#pragma unroll
            for (int c = 0; c < CPL; c++) {
                Elt<T>::widen(raw[u][c], f[c]);
#pragma unroll
                for (int i = 0; i < V; i++) s += f[c][i];
            }
            const float m = lanes_sum(s, d.lpg) * inv;
            s = 0.f;
#pragma unroll
            for (int c = 0; c < CPL; c++)
#pragma unroll
                for (int i = 0; i < V; i++) {
                    f[c][i] -= m;
                    if (has[c]) s = fmaf(f[c][i], f[c][i], s);
                }
            const float r = 1.0f / sqrtf(fmaf(lanes_sum(s, d.lpg), inv, eps));
            if (n >= d.N) continue;
#pragma unroll
            for (int c = 0; c < CPL; c++) {
#pragma unroll
                for (int i = 0; i < V; i++)
                    f[c][i] = activate<T, Silu>(fmaf(f[c][i] * r, wc[c][i], bc[c][i]));
                if (has[c])
                    st_stream(y + n * d.yn + t.at + c * d.lpg * V, Elt<T>::narrow(f[c]));
            }
            if (t.on && t.j == 0) {
                mean[n * d.G + t.g] = m;
                rstd[n * d.G + t.g] = r;
            }
        }
    }
    pdl_trigger();
}

template <typename T, int CPL, bool Silu>
__global__ void __launch_bounds__(RT, 2)
    gn_rows_bwd_kernel(const T* x, const T* dy, T* dx, const float* w, const float* b,
                       const float* mean, const float* rstd, float* part_a, float* part_b,
                       const RowShape d) {
    constexpr int V = Elt<T>::V, U = CPL == 1 ? 2 : 1;
    extern __shared__ float4 smem[];
    float* sum = reinterpret_cast<float*>(smem);  // [2][RW][CPL][V][32]
    const Place t(d, V);
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const float inv = 1.0f / (float)d.Cg;
    bool has[CPL];
    float wc[CPL][V], bc[CPL][V], A[CPL][V], B[CPL][V];
    pdl_wait();
#pragma unroll
    for (int c = 0; c < CPL; c++) {
        has[c] = t.on && t.j + c * d.lpg < d.cpg;
#pragma unroll
        for (int i = 0; i < V; i++) {
            wc[c][i] = has[c] ? __ldg(w + t.at + c * d.lpg * V + i) : 0.f;
            bc[c][i] = has[c] ? __ldg(b + t.at + c * d.lpg * V + i) : 0.f;
            A[c][i] = B[c][i] = 0.f;
        }
    }
    const int64_t step = (int64_t)d.RB * RW * d.rpw;
    const int64_t first = ((int64_t)(blockIdx.x / d.segs) * RW + wid) * d.rpw;
    for (int64_t n0 = first; n0 < d.N; n0 += U * step) {
        Raw16 rx[U][CPL], rg[U][CPL];
        float mu[U], rs[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            const int64_t n = n0 + u * step + t.sub;
            const bool in = t.on && n < d.N;
#pragma unroll
            for (int c = 0; c < CPL; c++) {
                const bool h = has[c] && n < d.N;
                const int64_t at = t.at + c * d.lpg * V;
                rx[u][c] = h ? ld_stream(x + n * d.xn + at) : raw_zero();
                rg[u][c] = h ? ld_stream(dy + n * d.gn + at) : raw_zero();
            }
            mu[u] = in ? mean[n * d.G + t.g] : 0.f;
            rs[u] = in ? rstd[n * d.G + t.g] : 0.f;
        }
#pragma unroll
        for (int u = 0; u < U; u++) {
            if (n0 + u * step >= d.N) break;
            const int64_t n = n0 + u * step + t.sub;
            float xh[CPL][V], g[CPL][V], m1 = 0.f, m2 = 0.f;
#pragma unroll
            for (int c = 0; c < CPL; c++) {
                Elt<T>::widen(rx[u][c], xh[c]);
                Elt<T>::widen(rg[u][c], g[c]);
#pragma unroll
                for (int i = 0; i < V; i++) {
                    // absent lanes hold zeros: dy = 0 keeps them out of every sum
                    xh[c][i] = (xh[c][i] - mu[u]) * rs[u];
                    const float dz = through<T, Silu>(g[c][i], fmaf(xh[c][i], wc[c][i], bc[c][i]));
                    A[c][i] = fmaf(dz, xh[c][i], A[c][i]);
                    B[c][i] += dz;
                    g[c][i] = dz * wc[c][i];
                    m1 += g[c][i];
                    m2 = fmaf(g[c][i], xh[c][i], m2);
                }
            }
            m1 = lanes_sum(m1, d.lpg) * inv;
            m2 = lanes_sum(m2, d.lpg) * inv;
            if (n >= d.N) continue;
#pragma unroll
            for (int c = 0; c < CPL; c++) {
#pragma unroll
                for (int i = 0; i < V; i++)
                    g[c][i] = rs[u] * (g[c][i] - m1 - xh[c][i] * m2);
                if (has[c])
                    st_stream(dx + n * d.yn + t.at + c * d.lpg * V, Elt<T>::narrow(g[c]));
            }
        }
    }
    // the block's sums, over its warps and a warp's rows in order
#pragma unroll
    for (int c = 0; c < CPL; c++)
#pragma unroll
        for (int i = 0; i < V; i++) {
            sum[((wid * CPL + c) * V + i) * 32 + lane] = A[c][i];
            sum[(((RW + wid) * CPL + c) * V + i) * 32 + lane] = B[c][i];
        }
    __syncthreads();
    if (t.on && t.sub == 0) {
        const int64_t row = (int64_t)(blockIdx.x / d.segs) * d.C;
        for (int e = wid; e < 2 * CPL * V; e += RW) {
            const int which = e / (CPL * V), c = e / V % CPL, i = e % V;
            if (t.j + c * d.lpg >= d.cpg) continue;
            float v = 0.f;
            for (int q = 0; q < RW; q++)
                for (int r = 0; r < d.rpw; r++)
                    v += sum[(((which * RW + q) * CPL + c) * V + i) * 32 + lane + r * d.spr];
            (which ? part_b : part_a)[row + t.at + c * d.lpg * V + i] = v;
        }
    }
    pdl_trigger();
}

// Row tiles of a sample: as many as give a chunk of samples about eight blocks
// an SM, of 16 KB to 256 KB each and at most 304 a sample (every block of the
// second pass reads its sample's tiles' statistics).  chunk: samples of one
// pair of passes, whose tensors (x, or x and dy) fit in L2.
constexpr int64_t kL2Chunk = 64 << 20;

Shape shape_of(int64_t N, int64_t S, int64_t C, int64_t G, int es, int tensors, int64_t& chunk) {
    Shape d{};
    d.S = S;
    d.C = (int)C;
    d.G = (int)G;
    d.Cg = (int)(C / G);
    const int64_t row = C * es, sample = S * row * tensors;
    chunk = std::min(N, std::max<int64_t>(1, kL2Chunk / sample));
    d.N = chunk;
    int64_t bytes = chunk * (S * row) / (kDesignSMs * 8);
    bytes = std::max<int64_t>(16 << 10, std::min<int64_t>(256 << 10, bytes));
    int64_t rows = std::max<int64_t>(1, bytes / row);
    rows = std::max(rows, (S + 303) / 304);
    const int64_t tiles = (S + rows - 1) / rows;
    d.rows = (S + tiles - 1) / tiles;
    d.tiles = (int)((S + d.rows - 1) / d.rows);
    return d;
}

// Blocks of the backward's first pass: rows of the channels' partial sums.
int64_t grad_rows(const Shape& d) {
    return std::min<int64_t>(d.N * d.tiles, kDesignSMs * 8);
}

int64_t pad64(int64_t n) { return (n + 63) / 64 * 64; }

size_t lanes_bytes(int C, int V) {
    const int cv = C / V;
    return (size_t)(cv < NT ? NT / cv : 1) * C * 4;
}

template <typename K>
cudaError_t allow(K kernel, size_t smem) {
    return smem <= 48 * 1024 ? cudaSuccess
                             : cudaFuncSetAttribute((const void*)kernel,
                                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    (int)smem);
}

// Whether S == 1 rows take the row kernels, and their shape: 16-byte vectors
// that no group shares, at most 64 of them a group.
bool row_shape(int64_t N, int64_t S, int64_t C, int64_t G, int es, RowShape& d) {
    const int V = 16 / es;
    const int64_t Cg = C / G;
    if (S != 1 || N == 0 || Cg % V || Cg / V > 64) return false;
    d = RowShape{};
    d.N = N;
    d.C = (int)C;
    d.G = (int)G;
    d.Cg = (int)Cg;
    d.cpg = (int)(Cg / V);
    const int cpl = d.cpg > 32 ? 2 : 1;
    d.lpg = 1;
    while (d.lpg * cpl < d.cpg) d.lpg *= 2;
    d.spr = d.G * d.lpg;
    d.rpw = d.spr < 32 ? 32 / d.spr : 1;
    d.segs = (d.spr + 31) / 32;
    // blocks along the samples: four an SM, fewer where warps would stand idle
    const int64_t per = (int64_t)RW * d.rpw, need = (N + per - 1) / per;
    const int64_t most = kDesignSMs * 4 / d.segs;
    d.RB = (int)(need < most ? need : most < 1 ? 1 : most);
    return true;
}

template <typename T, int CPL>
cudaError_t rows_fwd(const GroupNormFwd& a, const RowShape& d, bool silu, cudaStream_t s) {
    return launch(silu ? gn_rows_fwd_kernel<T, CPL, true> : gn_rows_fwd_kernel<T, CPL, false>,
                  dim3((unsigned)(d.segs * d.RB)), dim3(RT), 0, s, true, (const T*)a.x, (T*)a.y,
                  a.w, a.b, a.eps, a.mean, a.rstd, d);
}

template <typename T, int CPL>
cudaError_t rows_bwd(const GroupNormBwd& a, const RowShape& d, bool silu, cudaStream_t s) {
    float* pa = (float*)a.workspace;
    float* pb = pa + pad64((int64_t)d.RB * d.C);
    const auto k = silu ? gn_rows_bwd_kernel<T, CPL, true> : gn_rows_bwd_kernel<T, CPL, false>;
    const size_t smem = (size_t)2 * RW * CPL * Elt<T>::V * 32 * 4;
    cudaError_t e = allow(k, smem);
    if (e == cudaSuccess)
        e = launch(k, dim3((unsigned)(d.segs * d.RB)), dim3(RT), smem, s, true, (const T*)a.x,
                   (const T*)a.dy, (T*)a.dx, a.w, a.b, a.mean, a.rstd, pa, pb, d);
    if (e != cudaSuccess) return e;
    return launch(gn_grad_kernel, dim3((unsigned)((d.C + 31) / 32), 2), dim3(1024), 0, s, true,
                  (const float*)pa, (const float*)pb, (int64_t)d.RB, d.C, a.grad_w, a.grad_b,
                  a.accumulate);
}

template <typename T, int V>
cudaError_t fwd(const GroupNormFwd& a, Shape d, int64_t chunk, bool silu, cudaStream_t s) {
    float2* part = (float2*)a.workspace;
    const size_t smem = 2 * lanes_bytes(d.C, V), smem2 = (size_t)d.G * 8;
    const auto apply = silu ? gn_apply_kernel<T, V, true> : gn_apply_kernel<T, V, false>;
    cudaError_t e = allow(gn_stats_kernel<T, V>, smem);
    if (e == cudaSuccess) e = allow(apply, smem2);
    for (int64_t n = 0; n < a.N && e == cudaSuccess; n += chunk) {
        d.N = std::min(chunk, a.N - n);
        const dim3 grid((unsigned)(d.N * d.tiles));
        const T* x = (const T*)a.x + n * d.xn;
        e = launch(gn_stats_kernel<T, V>, grid, dim3(NT), smem, s, true, x, d, part);
        if (e == cudaSuccess)
            e = launch(apply, grid, dim3(NT), smem2, s, true, x, (T*)a.y + n * d.yn, a.w, a.b,
                       a.eps, a.mean + n * d.G, a.rstd + n * d.G, (const float2*)part, d);
    }
    return e;
}

template <typename T, int V>
cudaError_t bwd(const GroupNormBwd& a, Shape d, int64_t chunk, bool silu, cudaStream_t s) {
    const int64_t P = grad_rows(d), chunks = a.N ? (a.N + chunk - 1) / chunk : 0;
    float* pa = (float*)a.workspace;
    float* pb = pa + pad64(chunks * P * d.C);
    float2* pg = (float2*)(pb + pad64(chunks * P * d.C));
    const size_t smem = 2 * lanes_bytes(d.C, V), smem2 = (size_t)d.G * 16;
    const auto sums = silu ? gn_bwd_sums_kernel<T, V, true> : gn_bwd_sums_kernel<T, V, false>;
    const auto apply = silu ? gn_bwd_apply_kernel<T, V, true> : gn_bwd_apply_kernel<T, V, false>;
    cudaError_t e = allow(sums, smem);
    if (e == cudaSuccess) e = allow(apply, smem2);
    int64_t rows = 0;
    for (int64_t n = 0; n < a.N && e == cudaSuccess; n += chunk) {
        d.N = std::min(chunk, a.N - n);
        const int64_t p = grad_rows(d);
        const T *x = (const T*)a.x + n * d.xn, *dy = (const T*)a.dy + n * d.gn;
        const float *mean = a.mean + n * d.G, *rstd = a.rstd + n * d.G;
        e = launch(sums, dim3((unsigned)p), dim3(NT), smem, s, true, x, dy, a.w, a.b, mean, rstd, d,
                   pg, pa + rows * d.C, pb + rows * d.C);
        if (e == cudaSuccess)
            e = launch(apply, dim3((unsigned)(d.N * d.tiles)), dim3(NT), smem2, s, true, x, dy,
                       (T*)a.dx + n * d.yn, a.w, a.b, mean, rstd, (const float2*)pg, d);
        rows += p;
    }
    if (e != cudaSuccess) return e;
    return launch(gn_grad_kernel, dim3((unsigned)((d.C + 31) / 32), 2), dim3(1024), 0, s, true,
                  (const float*)pa, (const float*)pb, rows, d.C, a.grad_w, a.grad_b, a.accumulate);
}

}  // namespace

int64_t groupnorm_fwd_floats(int64_t N, int64_t S, int64_t C, int64_t G, int dtype) {
    if (N == 0 || S == 0 || C == 0) return 0;
    int64_t chunk;
    const Shape d = shape_of(N, S, C, G, elt_bytes(dtype), 1, chunk);
    return pad64(2 * chunk * d.tiles * G);
}

int64_t groupnorm_bwd_floats(int64_t N, int64_t S, int64_t C, int64_t G, int dtype) {
    if (N == 0 || S == 0 || C == 0) return 0;
    int64_t chunk;
    const Shape d = shape_of(N, S, C, G, elt_bytes(dtype), 2, chunk);
    const int64_t chunks = (N + chunk - 1) / chunk;
    int64_t n = 2 * pad64(chunks * grad_rows(d) * C) + pad64(2 * chunk * d.tiles * G);
    RowShape r;  // taken or not by the pointers' alignment
    if (row_shape(N, S, C, G, elt_bytes(dtype), r)) n = std::max(n, 2 * pad64((int64_t)r.RB * C));
    return n;
}

cudaError_t launch_groupnorm_fwd(const GroupNormFwd& a, cudaStream_t s) {
    const int es = elt_bytes(a.dtype);
    int64_t k;
    Shape d = shape_of(a.N, a.S, a.C, a.G, es, 1, k);
    d.xn = a.x_n, d.xs = a.x_s, d.yn = a.y_n, d.ys = a.y_s;
    const uint64_t bits = (uint64_t)a.C * es | (uint64_t)(uintptr_t)a.x | (uint64_t)(uintptr_t)a.y |
                          (a.N > 1 ? (uint64_t)(a.x_n | a.y_n) * es : 0) |
                          (a.S > 1 ? (uint64_t)(a.x_s | a.y_s) * es : 0);
    const bool vec = bits % 16 == 0, silu = a.act != 0;
    RowShape r;
    if (vec && row_shape(a.N, a.S, a.C, a.G, es, r)) {
        r.xn = a.x_n, r.yn = a.y_n;
        if (r.cpg > 32)
            return a.dtype == 0   ? rows_fwd<float, 2>(a, r, silu, s)
                   : a.dtype == 1 ? rows_fwd<__half, 2>(a, r, silu, s)
                                  : rows_fwd<__nv_bfloat16, 2>(a, r, silu, s);
        return a.dtype == 0   ? rows_fwd<float, 1>(a, r, silu, s)
               : a.dtype == 1 ? rows_fwd<__half, 1>(a, r, silu, s)
                              : rows_fwd<__nv_bfloat16, 1>(a, r, silu, s);
    }
    if (a.dtype == 0) return vec ? fwd<float, 4>(a, d, k, silu, s) : fwd<float, 1>(a, d, k, silu, s);
    if (a.dtype == 1) return vec ? fwd<__half, 8>(a, d, k, silu, s) : fwd<__half, 1>(a, d, k, silu, s);
    return vec ? fwd<__nv_bfloat16, 8>(a, d, k, silu, s) : fwd<__nv_bfloat16, 1>(a, d, k, silu, s);
}

cudaError_t launch_groupnorm_bwd(const GroupNormBwd& a, cudaStream_t s) {
    const int es = elt_bytes(a.dtype);
    if (a.N == 0 || a.S == 0)  // no values: the gradients' sums are empty
        return launch(gn_grad_kernel, dim3((unsigned)((a.C + 31) / 32), 2), dim3(1024), 0, s, true,
                      (const float*)nullptr, (const float*)nullptr, (int64_t)0, (int)a.C, a.grad_w,
                      a.grad_b, a.accumulate);
    int64_t k;
    Shape d = shape_of(a.N, a.S, a.C, a.G, es, 2, k);
    d.xn = a.x_n, d.xs = a.x_s, d.yn = a.dx_n, d.ys = a.dx_s, d.gn = a.dy_n, d.gs = a.dy_s;
    const uint64_t bits = (uint64_t)a.C * es | (uint64_t)(uintptr_t)a.x |
                          (uint64_t)(uintptr_t)a.dx | (uint64_t)(uintptr_t)a.dy |
                          (a.N > 1 ? (uint64_t)(a.x_n | a.dx_n | a.dy_n) * es : 0) |
                          (a.S > 1 ? (uint64_t)(a.x_s | a.dx_s | a.dy_s) * es : 0);
    const bool vec = bits % 16 == 0, silu = a.act != 0;
    RowShape r;
    if (vec && row_shape(a.N, a.S, a.C, a.G, es, r)) {
        r.xn = a.x_n, r.yn = a.dx_n, r.gn = a.dy_n;
        if (r.cpg > 32)
            return a.dtype == 0   ? rows_bwd<float, 2>(a, r, silu, s)
                   : a.dtype == 1 ? rows_bwd<__half, 2>(a, r, silu, s)
                                  : rows_bwd<__nv_bfloat16, 2>(a, r, silu, s);
        return a.dtype == 0   ? rows_bwd<float, 1>(a, r, silu, s)
               : a.dtype == 1 ? rows_bwd<__half, 1>(a, r, silu, s)
                              : rows_bwd<__nv_bfloat16, 1>(a, r, silu, s);
    }
    if (a.dtype == 0) return vec ? bwd<float, 4>(a, d, k, silu, s) : bwd<float, 1>(a, d, k, silu, s);
    if (a.dtype == 1) return vec ? bwd<__half, 8>(a, d, k, silu, s) : bwd<__half, 1>(a, d, k, silu, s);
    return vec ? bwd<__nv_bfloat16, 8>(a, d, k, silu, s) : bwd<__nv_bfloat16, 1>(a, d, k, silu, s);
}

}  // namespace wsf
