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

#include "wsf_block.h"
#include "wsf_device.cuh"
#include "wsf_internal.h"

namespace wsf {
namespace {

constexpr int NT = 512;

// V elements of T, read as binary32.
template <typename T, int V>
__device__ __forceinline__ void load_v(const T* p, float (&f)[V]) {
    if constexpr (V == 1)
        f[0] = Elt<T>::load1(p);
    else
        Elt<T>::widen(ld_keep(p), f);
}
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
    int64_t tiles, rows;  // row tiles of a sample, rows of a tile
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

// ---------------------------------------------------------------------------
// Mean and squared deviations of every group over one tile of a sample.
template <typename T, int V>
__global__ void __launch_bounds__(NT) gn_stats_kernel(const T* x, Shape d, float2* part) {
    extern __shared__ float4 smem[];
    const Lanes t(d.C, V);
    float* sm = reinterpret_cast<float*>(smem);  // [RL][C] means
    float* sq = sm + (size_t)t.RL * d.C;         // [RL][C] squared deviations
    pdl_wait();
    const int64_t n = blockIdx.x / d.tiles, tile = blockIdx.x - n * d.tiles;
    const int64_t s0 = tile * d.rows;
    const int rows = (int)min(d.rows, d.S - s0);
    const T* base = x + n * d.xn + s0 * d.xs;
    if (t.r < t.RL) {
        for (int c = t.c; c < t.cv; c += NT) {
            float k[V], a[V], b[V];
#pragma unroll
            for (int i = 0; i < V; i++) k[i] = a[i] = b[i] = 0.f;
            const int cnt = t.r < rows ? (rows - t.r + t.RL - 1) / t.RL : 0;
            const T* p = base + (int64_t)t.r * d.xs + c * V;
            if (cnt) {
                load_v<T, V>(p, k);
#pragma unroll 4
                for (int j = 1; j < cnt; j++) {
                    float f[V];
                    load_v<T, V>(p + (int64_t)j * t.RL * d.xs, f);
#pragma unroll
                    for (int i = 0; i < V; i++) {
                        const float q = f[i] - k[i];
                        a[i] += q;
                        b[i] = fmaf(q, q, b[i]);
                    }
                }
            }
            const float inv = cnt ? 1.0f / cnt : 0.f;
#pragma unroll
            for (int i = 0; i < V; i++) {
                const float m = a[i] * inv;
                sm[t.r * d.C + c * V + i] = k[i] + m;
                sq[t.r * d.C + c * V + i] = fmaxf(fmaf(-m, a[i], b[i]), 0.f);
            }
        }
    }
    __syncthreads();
    // a warp joins a group: RL x Cg entries, row lane r standing for cnt(r) rows
    const int lane = threadIdx.x & 31;
    const float inv = 1.0f / ((float)rows * d.Cg);
    for (int g = threadIdx.x >> 5; g < d.G; g += NT / 32) {
        float s = 0.f;
        for (int e = lane; e < t.RL * d.Cg; e += 32) {
            const int r = e / d.Cg, at = r * d.C + g * d.Cg + e - r * d.Cg;
            const int cnt = r < rows ? (rows - r + t.RL - 1) / t.RL : 0;
            s = fmaf((float)cnt, sm[at], s);
        }
        const float mean = group_sum<32>(s) * inv;
        s = 0.f;
        for (int e = lane; e < t.RL * d.Cg; e += 32) {
            const int r = e / d.Cg, at = r * d.C + g * d.Cg + e - r * d.Cg;
            const int cnt = r < rows ? (rows - r + t.RL - 1) / t.RL : 0;
            const float q = sm[at] - mean;
            if (cnt) s += fmaf((float)cnt * q, q, sq[at]);
        }
        s = group_sum<32>(s);
        if (lane == 0) part[(int64_t)blockIdx.x * d.G + g] = make_float2(mean, s);
    }
    pdl_trigger();
}

// A warp a (sample, group): the tiles' statistics joined.
__global__ void __launch_bounds__(256) gn_join_kernel(const float2* part, Shape d, float eps,
                                                      float* mean, float* rstd) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (u < d.N * d.G) {
        const int64_t n = u / d.G, g = u - n * d.G;
        const float2* p = part + n * d.tiles * d.G + g;
        const float inv = 1.0f / (float)d.S;
        float s = 0.f;
        for (int64_t i = lane; i < d.tiles; i += 32)
            s = fmaf((float)min(d.rows, d.S - i * d.rows), p[i * d.G].x, s);
        const float m = group_sum<32>(s) * inv;
        s = 0.f;
        for (int64_t i = lane; i < d.tiles; i += 32) {
            const float2 q = p[i * d.G];
            const float w = (float)min(d.rows, d.S - i * d.rows) * d.Cg, e = q.x - m;
            s += fmaf(w * e, e, q.y);
        }
        s = group_sum<32>(s);
        if (lane == 0) {
            mean[u] = m;
            rstd[u] = 1.0f / sqrtf(s / ((float)d.S * d.Cg) + eps);
        }
    }
    pdl_trigger();
}

template <typename T, int V, bool Silu>
__global__ void __launch_bounds__(NT) gn_apply_kernel(const T* x, T* y, const float* w,
                                                      const float* b, const float* mean,
                                                      const float* rstd, Shape d) {
    const Lanes t(d.C, V);
    pdl_wait();
    const int64_t n = blockIdx.x / d.tiles, tile = blockIdx.x - n * d.tiles;
    const int64_t s0 = tile * d.rows;
    const int rows = (int)min(d.rows, d.S - s0);
    if (t.r < t.RL) {
        for (int c = t.c; c < t.cv; c += NT) {
            float mu[V], rw[V], sh[V];
#pragma unroll
            for (int i = 0; i < V; i++) {
                const int ch = c * V + i;
                const int64_t g = n * d.G + ch / d.Cg;
                mu[i] = mean[g];
                rw[i] = rstd[g] * __ldg(w + ch);
                sh[i] = __ldg(b + ch);
            }
#pragma unroll 4
            for (int s = t.r; s < rows; s += t.RL) {
                float f[V];
                load_v<T, V>(x + n * d.xn + (s0 + s) * d.xs + c * V, f);
#pragma unroll
                for (int i = 0; i < V; i++)
                    f[i] = activate<T, Silu>(fmaf(f[i] - mu[i], rw[i], sh[i]));
                store_v<T, V>(y + n * d.yn + (s0 + s) * d.ys + c * V, f);
            }
        }
    }
    pdl_trigger();
}

// ---------------------------------------------------------------------------
// Backward, first pass: a block walks units (sample, tile) u0 .. u1 and
// writes each unit's groups' sums (m₂, m₁ shares) and, over all of them, the
// channels' sums.
template <typename T, int V, bool Silu>
__global__ void __launch_bounds__(NT) gn_bwd_sums_kernel(const T* x, const T* dy, const float* w,
                                                         const float* b, const float* mean,
                                                         const float* rstd, Shape d, float2* part_g,
                                                         float* part_a, float* part_b) {
    extern __shared__ float4 smem[];
    const Lanes t(d.C, V);
    float* sa = reinterpret_cast<float*>(smem);  // [RL][C]
    float* sb = sa + (size_t)t.RL * d.C;         // [RL][C]
    float* ta = part_a + (int64_t)blockIdx.x * d.C;  // [C] the block's own row
    float* tb = part_b + (int64_t)blockIdx.x * d.C;
    pdl_wait();
    const int64_t units = d.N * d.tiles;
    const int64_t u0 = units * blockIdx.x / gridDim.x, u1 = units * (blockIdx.x + 1) / gridDim.x;
    for (int64_t u = u0; u < u1; u++) {
        const int64_t n = u / d.tiles, tile = u - n * d.tiles, s0 = tile * d.rows;
        const int rows = (int)min(d.rows, d.S - s0);
        if (t.r < t.RL) {
            for (int c = t.c; c < t.cv; c += NT) {
                float mu[V], rs[V], wc[V], bc[V], A[V], B[V];
#pragma unroll
                for (int i = 0; i < V; i++) {
                    const int ch = c * V + i;
                    const int64_t g = n * d.G + ch / d.Cg;
                    mu[i] = mean[g];
                    rs[i] = rstd[g];
                    wc[i] = __ldg(w + ch);
                    bc[i] = __ldg(b + ch);
                    A[i] = B[i] = 0.f;
                }
#pragma unroll 2
                for (int s = t.r; s < rows; s += t.RL) {
                    float f[V], g[V];
                    load_v<T, V>(x + n * d.xn + (s0 + s) * d.xs + c * V, f);
                    load_v<T, V>(dy + n * d.gn + (s0 + s) * d.gs + c * V, g);
#pragma unroll
                    for (int i = 0; i < V; i++) {
                        const float xh = (f[i] - mu[i]) * rs[i];
                        const float dz = through<T, Silu>(g[i], fmaf(xh, wc[i], bc[i]));
                        A[i] = fmaf(dz, xh, A[i]);
                        B[i] += dz;
                    }
                }
#pragma unroll
                for (int i = 0; i < V; i++) {
                    sa[t.r * d.C + c * V + i] = A[i];
                    sb[t.r * d.C + c * V + i] = B[i];
                }
            }
        }
        __syncthreads();
        for (int c = threadIdx.x; c < d.C; c += NT) {  // over the row lanes, in order
            float A = sa[c], B = sb[c];
            for (int r = 1; r < t.RL; r++) A += sa[r * d.C + c], B += sb[r * d.C + c];
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

// A warp a (sample, group): m₂ and m₁ over the tiles.
__global__ void __launch_bounds__(256) gn_bwd_join_kernel(const float2* part, Shape d, float2* m) {
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    if (u < d.N * d.G) {
        const int64_t n = u / d.G, g = u - n * d.G;
        const float2* p = part + n * d.tiles * d.G + g;
        float A = 0.f, B = 0.f;
        for (int64_t i = lane; i < d.tiles; i += 32) {
            const float2 q = p[i * d.G];
            A += q.x;
            B += q.y;
        }
        A = group_sum<32>(A);
        B = group_sum<32>(B);
        const float inv = 1.0f / ((float)d.S * d.Cg);
        if (lane == 0) m[u] = make_float2(A * inv, B * inv);
    }
    pdl_trigger();
}

template <typename T, int V, bool Silu>
__global__ void __launch_bounds__(NT) gn_bwd_apply_kernel(const T* x, const T* dy, T* dx,
                                                          const float* w, const float* b,
                                                          const float* mean, const float* rstd,
                                                          const float2* m, Shape d) {
    const Lanes t(d.C, V);
    pdl_wait();
    const int64_t n = blockIdx.x / d.tiles, tile = blockIdx.x - n * d.tiles;
    const int64_t s0 = tile * d.rows;
    const int rows = (int)min(d.rows, d.S - s0);
    if (t.r < t.RL) {
        for (int c = t.c; c < t.cv; c += NT) {
            float mu[V], rs[V], wc[V], bc[V], m2[V], m1[V];
#pragma unroll
            for (int i = 0; i < V; i++) {
                const int ch = c * V + i;
                const int64_t g = n * d.G + ch / d.Cg;
                mu[i] = mean[g];
                rs[i] = rstd[g];
                wc[i] = __ldg(w + ch);
                bc[i] = __ldg(b + ch);
                const float2 q = m[g];
                m2[i] = q.x;
                m1[i] = q.y;
            }
#pragma unroll 2
            for (int s = t.r; s < rows; s += t.RL) {
                float f[V], g[V];
                load_v<T, V>(x + n * d.xn + (s0 + s) * d.xs + c * V, f);
                load_v<T, V>(dy + n * d.gn + (s0 + s) * d.gs + c * V, g);
#pragma unroll
                for (int i = 0; i < V; i++) {
                    const float xh = (f[i] - mu[i]) * rs[i];
                    const float dz = through<T, Silu>(g[i], fmaf(xh, wc[i], bc[i]));
                    f[i] = rs[i] * (fmaf(dz, wc[i], -m1[i]) - xh * m2[i]);
                }
                store_v<T, V>(dx + n * d.yn + (s0 + s) * d.ys + c * V, f);
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

// Row tiles: about 64 KB of x each.
Shape shape_of(int64_t N, int64_t S, int64_t C, int64_t G, int es) {
    Shape d{};
    d.N = N;
    d.S = S;
    d.C = (int)C;
    d.G = (int)G;
    d.Cg = (int)(C / G);
    int64_t rows = 65536 / (C * es);
    if (rows < 1) rows = 1;
    int64_t tiles = (S + rows - 1) / rows;
    d.rows = (S + tiles - 1) / tiles;
    d.tiles = (S + d.rows - 1) / d.rows;
    return d;
}

int64_t grad_rows(const Shape& d) {
    const int64_t u = d.N * d.tiles;
    return u < kDesignSMs * 2 ? u : kDesignSMs * 2;
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

template <typename T, int V>
cudaError_t fwd(const GroupNormFwd& a, const Shape& d, bool silu, cudaStream_t s) {
    float2* part = (float2*)a.workspace;
    const unsigned units = (unsigned)(d.N * d.tiles);
    const size_t smem = 2 * lanes_bytes(d.C, V);
    cudaError_t e = allow(gn_stats_kernel<T, V>, smem);
    if (e == cudaSuccess)
        e = launch(gn_stats_kernel<T, V>, dim3(units), dim3(NT), smem, s, true, (const T*)a.x, d,
                   part);
    if (e == cudaSuccess)
        e = launch(gn_join_kernel, dim3((unsigned)((d.N * d.G + 7) / 8)), dim3(256), 0, s, true,
                   (const float2*)part, d, a.eps, a.mean, a.rstd);
    if (e != cudaSuccess) return e;
    return launch(silu ? gn_apply_kernel<T, V, true> : gn_apply_kernel<T, V, false>, dim3(units),
                  dim3(NT), 0, s, true, (const T*)a.x, (T*)a.y, a.w, a.b, (const float*)a.mean,
                  (const float*)a.rstd, d);
}

template <typename T, int V>
cudaError_t bwd(const GroupNormBwd& a, const Shape& d, bool silu, cudaStream_t s) {
    const int64_t units = d.N * d.tiles, P = grad_rows(d);
    float* pa = (float*)a.workspace;
    float* pb = pa + pad64(P * d.C);
    float2* pg = (float2*)(pb + pad64(P * d.C));
    float2* m = pg + pad64(units * d.G);
    cudaError_t e = cudaSuccess;
    if (units > 0) {
        const size_t smem = 2 * lanes_bytes(d.C, V);
        const auto sums = silu ? gn_bwd_sums_kernel<T, V, true> : gn_bwd_sums_kernel<T, V, false>;
        e = allow(sums, smem);
        if (e == cudaSuccess)
            e = launch(sums, dim3((unsigned)P), dim3(NT), smem, s, true, (const T*)a.x,
                       (const T*)a.dy, a.w, a.b, a.mean, a.rstd, d, pg, pa, pb);
        if (e == cudaSuccess)
            e = launch(gn_bwd_join_kernel, dim3((unsigned)((d.N * d.G + 7) / 8)), dim3(256), 0, s,
                       true, (const float2*)pg, d, m);
        if (e == cudaSuccess)
            e = launch(silu ? gn_bwd_apply_kernel<T, V, true> : gn_bwd_apply_kernel<T, V, false>,
                       dim3((unsigned)units), dim3(NT), 0, s, true, (const T*)a.x, (const T*)a.dy,
                       (T*)a.dx, a.w, a.b, a.mean, a.rstd, (const float2*)m, d);
        if (e != cudaSuccess) return e;
    }
    return launch(gn_grad_kernel, dim3((unsigned)((d.C + 31) / 32), 2), dim3(1024), 0, s, true,
                  (const float*)pa, (const float*)pb, units > 0 ? P : (int64_t)0, d.C, a.grad_w,
                  a.grad_b, a.accumulate);
}

}  // namespace

int64_t groupnorm_fwd_floats(int64_t N, int64_t S, int64_t C, int64_t G, int dtype) {
    if (N == 0 || S == 0 || C == 0) return 0;
    const Shape d = shape_of(N, S, C, G, elt_bytes(dtype));
    return pad64(2 * d.N * d.tiles * d.G);
}

int64_t groupnorm_bwd_floats(int64_t N, int64_t S, int64_t C, int64_t G, int dtype) {
    if (N == 0 || S == 0 || C == 0) return 0;
    const Shape d = shape_of(N, S, C, G, elt_bytes(dtype));
    return 2 * pad64(grad_rows(d) * d.C) + 2 * pad64(d.N * d.tiles * d.G) + pad64(2 * d.N * d.G);
}

int64_t groupnorm_units(int64_t N, int64_t S, int64_t C, int64_t G, int dtype) {
    return N == 0 || S == 0 || C == 0 ? 0 : N * shape_of(N, S, C, G, elt_bytes(dtype)).tiles;
}

cudaError_t launch_groupnorm_fwd(const GroupNormFwd& a, cudaStream_t s) {
    const int es = elt_bytes(a.dtype);
    Shape d = shape_of(a.N, a.S, a.C, a.G, es);
    d.xn = a.x_n, d.xs = a.x_s, d.yn = a.y_n, d.ys = a.y_s;
    const uint64_t bits = (uint64_t)a.C * es | (uint64_t)(uintptr_t)a.x | (uint64_t)(uintptr_t)a.y |
                          (a.N > 1 ? (uint64_t)(a.x_n | a.y_n) * es : 0) |
                          (a.S > 1 ? (uint64_t)(a.x_s | a.y_s) * es : 0);
    const bool vec = bits % 16 == 0, silu = a.act != 0;
    if (a.dtype == 0) return vec ? fwd<float, 4>(a, d, silu, s) : fwd<float, 1>(a, d, silu, s);
    if (a.dtype == 1) return vec ? fwd<__half, 8>(a, d, silu, s) : fwd<__half, 1>(a, d, silu, s);
    return vec ? fwd<__nv_bfloat16, 8>(a, d, silu, s) : fwd<__nv_bfloat16, 1>(a, d, silu, s);
}

cudaError_t launch_groupnorm_bwd(const GroupNormBwd& a, cudaStream_t s) {
    const int es = elt_bytes(a.dtype);
    Shape d = a.N > 0 && a.S > 0 ? shape_of(a.N, a.S, a.C, a.G, es) : Shape{};
    d.C = (int)a.C;
    d.xn = a.x_n, d.xs = a.x_s, d.yn = a.dx_n, d.ys = a.dx_s, d.gn = a.dy_n, d.gs = a.dy_s;
    const uint64_t bits = (uint64_t)a.C * es | (uint64_t)(uintptr_t)a.x |
                          (uint64_t)(uintptr_t)a.dx | (uint64_t)(uintptr_t)a.dy |
                          (a.N > 1 ? (uint64_t)(a.x_n | a.dx_n | a.dy_n) * es : 0) |
                          (a.S > 1 ? (uint64_t)(a.x_s | a.dx_s | a.dy_s) * es : 0);
    const bool vec = bits % 16 == 0, silu = a.act != 0;
    if (a.dtype == 0) return vec ? bwd<float, 4>(a, d, silu, s) : bwd<float, 1>(a, d, silu, s);
    if (a.dtype == 1) return vec ? bwd<__half, 8>(a, d, silu, s) : bwd<__half, 1>(a, d, silu, s);
    return vec ? bwd<__nv_bfloat16, 8>(a, d, silu, s) : bwd<__nv_bfloat16, 1>(a, d, silu, s);
}

}  // namespace wsf
