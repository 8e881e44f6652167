// router.cu — the top-k router of a mixture of experts (sm_103a): softmax
// gates of the k largest logits of each row, per-expert counts and the
// balance loss, and their vector-Jacobian product.
//
//   p = softmax(l),  ids = the k largest logits, equal ones in index order
//   gates_j = p[ids_j]   or   p[ids_j] / Σ_i p[ids_i]
//   loss = E·Σ_e (c_e / kV)·(Σ_t p_te / V),   V = rows that count
//
// with c the counts.  The choice and the counts are constants of the
// backward, so with a_e = dloss·E·c_e/(k·V²) and u the gates' gradient put
// at the chosen experts
//   dl = p·(g − Σ g·p),  g = a + u                     (plain gates)
//   dl = p·(a − Σ a·p) + [e chosen] gate·(u − Σ u·gate)  (normalised gates)
//
// A row is held by L lanes (8 consecutive experts a lane; rows wider than
// 256 experts give each lane 2 or 4 such runs), 32/L rows a warp, so that
// reductions over a row are log2 L shuffles shared by all of a warp's rows.
// The k largest are taken one at a time: each lane's maximum of
// order-preserving integer keys, a butterfly over the row's lanes, and the
// winner's key cleared.  For 16-bit storage a key holds the value's 16 bits
// above the complement of the expert's index, so that one integer maximum
// also settles ties; binary32 carries the index beside the key.  The largest
// is also the softmax's shift.
//
// Σ_t p_te is summed in registers (every lane keeps its experts for all
// rows), then over the block, into one partial row a block; a second kernel
// adds the partial rows in a fixed order.  Counts are integers, exact in any
// order.
#include <stdint.h>

#include <type_traits>

#include "wsf_block.h"
#include "wsf_device.cuh"
#include "wsf_internal.h"

namespace wsf {
namespace {

constexpr int NW = 8;            // warps of a block
constexpr int NT = NW * 32;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ninf() { return __int_as_float(0xff800000); }

// 2^x by the hardware's exponential (about 2 units in the last place).
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// exp(f − m).  The difference is taken first: m·log₂ e alone overflows where
// every logit is the type's lowest value.
__device__ __forceinline__ float exp_of(float f, float m) { return ex2((f - m) * kLog2e); }

// Integers in the order of the values (−0 as +0, NaN at the ends); 0 stands
// for an expert that is taken or does not exist.  For 16-bit storage the low
// half is the complement of the expert's index e < 2¹⁶ − 1.
template <typename T>
__device__ __forceinline__ uint32_t order_key(float f, int e) {
    if constexpr (sizeof(T) == 4) {
        const uint32_t b = __float_as_uint(f + 0.0f);
        return max(b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u), 1u);
    } else {
        uint32_t b;
        if constexpr (std::is_same<T, __half>::value)
            b = (uint32_t)__half_as_ushort(__float2half_rn(f + 0.0f)) << 16;
        else
            b = __float_as_uint(f + 0.0f);
        b ^= (uint32_t)((int32_t)b >> 31) | 0x80000000u;
        return (b & 0xffff0000u) | (uint32_t)(0xffff - e);
    }
}

// The value an order_key stands for.
template <typename T>
__device__ __forceinline__ float key_value(uint32_t key) {
    uint32_t b = key ^ (~(uint32_t)((int32_t)key >> 31) | 0x80000000u);
    if constexpr (sizeof(T) == 4)
        return __uint_as_float(b);
    else if constexpr (std::is_same<T, __half>::value)
        return __half2float(__ushort_as_half((unsigned short)(b >> 16)));
    else
        return __uint_as_float(b & 0xffff0000u);
}

// Index of element i of a lane's 8·R experts.
template <int L>
__device__ __forceinline__ int expert(int i, int sub) {
    return ((i / 8) * L + sub) * 8 + i % 8;
}

// The lane's 8·R logits of a row as binary32, −inf behind the last expert.
// Rows of experts in eights at 16-byte addresses (vec) are read and written
// 16 bytes at a time, others element by element.
template <typename T, int L, int R>
__device__ __forceinline__ void load_row(const T* row, bool on, int sub, int E, bool vec,
                                         float (&f)[8 * R]) {
    constexpr int V = Elt<T>::V;
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int e0 = expert<L>(r * 8, sub);
        if (vec) {
#pragma unroll
            for (int h = 0; h < 8; h += V) {
                float g[V];
                if (on && e0 < E) {
                    Elt<T>::widen(ld_keep(row + e0 + h), g);
                } else {
#pragma unroll
                    for (int i = 0; i < V; i++) g[i] = ninf();
                }
#pragma unroll
                for (int i = 0; i < V; i++) f[r * 8 + h + i] = g[i];
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                f[r * 8 + i] = on && e0 + i < E ? Elt<T>::load1(row + e0 + i) : ninf();
        }
    }
}

template <typename T, int L, int R>
__device__ __forceinline__ void store_row(T* row, int sub, int E, bool vec,
                                          const float (&f)[8 * R]) {
    constexpr int V = Elt<T>::V;
#pragma unroll
    for (int r = 0; r < R; r++) {
        const int e0 = expert<L>(r * 8, sub);
        if (vec) {
#pragma unroll
            for (int h = 0; h < 8; h += V) {
                float g[V];
#pragma unroll
                for (int i = 0; i < V; i++) g[i] = f[r * 8 + h + i];
                if (e0 < E) st_stream(row + e0 + h, Elt<T>::narrow(g));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; i++)
                if (e0 + i < E) Elt<T>::store1(row + e0 + i, f[r * 8 + i]);
        }
    }
}

// ---------------------------------------------------------------------------
struct FwdArgs {
    const void* logits;
    const unsigned char* mask;
    float* gates;
    int* ids;
    float* part_p;  // [P, E]
    int* part_c;    // [P, E]
    int64_t ld;
    int64_t T;
    int E, k, renorm, vec;
};

template <int L, int R>
size_t fwd_smem(int k) {
    return (size_t)(NW + 1) * L * 8 * R * 4 + (size_t)NW * (32 / L) * k * 8;
}

template <typename T, int L, int R>
__global__ void __launch_bounds__(NT) router_fwd_kernel(const FwdArgs a) {
    constexpr int EPL = 8 * R, RPW = 32 / L, SLOTS = L * EPL;
    extern __shared__ float4 smem4[];
    float* ps = reinterpret_cast<float*>(smem4);             // [NW][SLOTS]
    int* cnt = reinterpret_cast<int*>(ps + NW * SLOTS);      // [SLOTS]
    float2* took = reinterpret_cast<float2*>(cnt + SLOTS);   // [NW][RPW][k]: value, expert
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int sub = lane & (L - 1), grp = lane / L;
    const int E = a.E, k = a.k;
    float2* mine = took + (wid * RPW + grp) * k;

    for (int i = threadIdx.x; i < SLOTS; i += NT) cnt[i] = 0;
    __syncthreads();
    pdl_wait();
    float sum_p[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) sum_p[i] = 0.f;

    const int64_t step = (int64_t)gridDim.x * NW * RPW;
    for (int64_t row0 = ((int64_t)blockIdx.x * NW + wid) * RPW; row0 < a.T; row0 += step) {
        const int64_t row = row0 + grp;
        const bool on = row < a.T;
        float f[EPL];
        load_row<T, L, R>((const T*)a.logits + row * a.ld, on, sub, E, a.vec, f);
        bool valid = on && (!a.mask || a.mask[row]);

        // the k largest, in order
        uint32_t key[EPL];
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const int e = expert<L>(i, sub);
            key[i] = e < E ? order_key<T>(f[i], e) : 0u;
        }
        float m = 0.f;
        for (int j = 0; j < k; j++) {
            uint32_t best = key[0];
            int id;
            if constexpr (sizeof(T) == 2) {
#pragma unroll
                for (int i = 1; i < EPL; i++) best = max(best, key[i]);
                if constexpr (L == 32) {
                    best = __reduce_max_sync(FULL_MASK, best);
                } else {
#pragma unroll
                    for (int o = L / 2; o > 0; o >>= 1)
                        best = max(best, __shfl_xor_sync(FULL_MASK, best, o));
                }
#pragma unroll
                for (int i = 0; i < EPL; i++) key[i] = key[i] == best ? 0u : key[i];
                id = 0xffff - (int)(best & 0xffffu);
            } else {
                id = expert<L>(0, sub);
#pragma unroll
                for (int i = 1; i < EPL; i++) {
                    const bool up = key[i] > best;  // in index order: a tie keeps the first
                    best = up ? key[i] : best;
                    id = up ? expert<L>(i, sub) : id;
                }
#pragma unroll
                for (int o = L / 2; o > 0; o >>= 1) {
                    const uint32_t ob = __shfl_xor_sync(FULL_MASK, best, o);
                    const int oi = __shfl_xor_sync(FULL_MASK, id, o);
                    const bool up = ob > best || (ob == best && oi < id);
                    best = up ? ob : best;
                    id = up ? oi : id;
                }
#pragma unroll
                for (int i = 0; i < EPL; i++)
                    key[i] = expert<L>(i, sub) == id ? 0u : key[i];
            }
            const float v = key_value<T>(best);
            if (j == 0) m = v;
            if (sub == 0) mine[j] = make_float2(v, __int_as_float(id));
        }
        valid = valid && m != ninf();  // no logit above −inf: the row does not count

        // softmax, shifted by the largest
        m = valid ? m : 0.f;
        float z = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            f[i] = exp_of(f[i], m);
            z += f[i];
        }
        z = group_sum<L>(z);
        if (valid) {
            const float inv = 1.0f / z;
#pragma unroll
            for (int i = 0; i < EPL; i++) sum_p[i] = fmaf(f[i], inv, sum_p[i]);
        }

        // gates and ids, in the order of memory
        __syncwarp();
        if (a.renorm) {
            z = 0.f;
            for (int j = sub; j < k; j += L) z += exp_of(mine[j].x, m);
            z = group_sum<L>(z);
        }
        if (on) {
            for (int j = sub; j < k; j += L) {
                const float2 q = mine[j];
                const int id = __float_as_int(q.y);
                a.gates[row * k + j] = valid ? exp_of(q.x, m) / z : 0.f;
                a.ids[row * k + j] = valid ? id : -1;
                if (valid) atomicAdd(&cnt[id], 1);
            }
        }
        __syncwarp();
    }

    // the block's sums: over the warp's rows, then over the warps in order
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        float v = sum_p[i];
#pragma unroll
        for (int o = L; o < 32; o <<= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
        if (grp == 0) ps[wid * SLOTS + expert<L>(i, sub)] = v;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += NT) {
        float v = ps[e];
#pragma unroll
        for (int w = 1; w < NW; w++) v += ps[w * SLOTS + e];
        a.part_p[(int64_t)blockIdx.x * E + e] = v;
        a.part_c[(int64_t)blockIdx.x * E + e] = cnt[e];
    }
    pdl_trigger();
}

// counts, and the loss, from the P partial rows: column e is summed by 32
// threads (rows p ≡ stripe mod 32 in order, then a fixed butterfly).  The
// grid is one cluster; CTA 0 adds the CTAs' shares of the loss.  c·S is
// formed and summed in binary64: at most 1024 terms.
constexpr int RT = 1024;

__global__ void __launch_bounds__(RT) router_reduce_kernel(const float* part_p, const int* part_c,
                                                           int P, int E, int k, int* counts,
                                                           float* loss) {
    __shared__ double share[RT / 32];
    __shared__ long long chose[RT / 32];
    __shared__ double all_share[8];
    __shared__ long long all_chose[8];
    pdl_wait();
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const unsigned me = cluster_ctarank(), cs = cluster_nctarank();
    double sh = 0.0;
    long long ch = 0;
    for (int e = me * (RT / 32) + wid; e < E; e += cs * (RT / 32)) {
        Acc2 s = acc2_zero();
        int c = 0;
        for (int p = lane; p < P; p += 32) {
            acc2_add1(s, __ldg(part_p + (int64_t)p * E + e));
            c += __ldg(part_c + (int64_t)p * E + e);
        }
        s = group_sum2<32>(s);
        c = __reduce_add_sync(FULL_MASK, c);
        if (lane == 0) counts[e] = c;
        sh += (double)c * ((double)s.hi + (double)s.lo);
        ch += c;
    }
    if (lane == 0) share[wid] = sh, chose[wid] = ch;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int w = 1; w < RT / 32; w++) sh += share[w], ch += chose[w];
        const uint32_t ds = cluster_map(&all_share[me], 0), dc = cluster_map(&all_chose[me], 0);
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(ds), "d"(sh) : "memory");
        asm volatile("st.shared::cluster.s64 [%0], %1;" ::"r"(dc), "l"(ch) : "memory");
    }
    cluster_sync();
    if (me == 0 && threadIdx.x == 0) {
        sh = 0.0, ch = 0;
        for (unsigned r = 0; r < cs; r++) sh += all_share[r], ch += all_chose[r];
        // V = ch / k rows count: loss = E·Σ c·S / (k·V²) = E·k·Σ c·S / ch²
        *loss = ch ? (float)((double)E * k * sh / ((double)ch * (double)ch)) : 0.f;
    }
    pdl_trigger();
}

// ---------------------------------------------------------------------------
struct BwdArgs {
    const void* logits;
    const int* ids;
    const int* counts;
    const float* dgates;
    const float* dloss;
    void* dlogits;
    int64_t ld, ldd;
    int64_t T;
    int E, k, renorm, vec;
};

template <int L, int R>
size_t bwd_smem() {
    return (size_t)NW * 32 * 8 * R * 4 + 64;
}

template <typename T, int L, int R>
__global__ void __launch_bounds__(NT) router_bwd_kernel(const BwdArgs a) {
    constexpr int EPL = 8 * R, RPW = 32 / L, SLOTS = L * EPL;
    extern __shared__ float4 smem4[];
    float* put = reinterpret_cast<float*>(smem4);  // [NW][RPW][SLOTS]: gradients at their experts
    long long* tot = reinterpret_cast<long long*>(put + NW * RPW * SLOTS);  // [NW]
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int sub = lane & (L - 1), grp = lane / L;
    const int E = a.E, k = a.k;
    float* mine = put + (wid * RPW + grp) * SLOTS;
    for (int i = threadIdx.x; i < NW * RPW * SLOTS; i += NT) put[i] = 0.f;
    pdl_wait();
    long long ch = 0;
    for (int e = threadIdx.x; e < E; e += NT) ch += a.counts[e];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ch += __shfl_xor_sync(FULL_MASK, ch, o);
    if (lane == 0) tot[wid] = ch;
    __syncthreads();
    ch = 0;
#pragma unroll
    for (int w = 0; w < NW; w++) ch += tot[w];
    // a_e = dloss·E·c_e/(k·V²) = dloss·E·k·c_e/ch²
    const float V = (float)ch / k;
    const float unit = ch > 0 && a.dloss ? *a.dloss * ((float)E / (k * V)) / V : 0.f;
    float ae[EPL];
#pragma unroll
    for (int i = 0; i < EPL; i++) {
        const int e = expert<L>(i, sub);
        ae[i] = e < E ? unit * (float)a.counts[e] : 0.f;
    }

    const int64_t step = (int64_t)gridDim.x * NW * RPW;
    for (int64_t row0 = ((int64_t)blockIdx.x * NW + wid) * RPW; row0 < a.T; row0 += step) {
        const int64_t row = row0 + grp;
        const bool on = row < a.T;
        const T* src = (const T*)a.logits + row * a.ld;
        float f[EPL];
        load_row<T, L, R>(src, on, sub, E, a.vec, f);
        const int* ids = a.ids + row * k;
        const bool valid = on && ids[0] >= 0;
        float m = f[0];
#pragma unroll
        for (int i = 1; i < EPL; i++) m = fmaxf(m, f[i]);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(FULL_MASK, m, o));
        m = valid ? m : 0.f;

        // the gates' gradient, at its experts
        const bool put_u = valid && a.dgates;
        if (a.renorm) {
            float zs = 0.f, dot = 0.f;
            if (put_u)
                for (int j = sub; j < k; j += L) {
                    const unsigned id = ids[j];
                    if (id >= (unsigned)E) continue;
                    const float e = exp_of(Elt<T>::load1(src + id), m);
                    zs += e;
                    dot = fmaf(e, a.dgates[row * k + j], dot);
                }
            zs = group_sum<L>(zs);
            dot = group_sum<L>(dot) / zs;
            if (put_u)
                for (int j = sub; j < k; j += L) {
                    const unsigned id = ids[j];
                    if (id >= (unsigned)E) continue;
                    const float e = exp_of(Elt<T>::load1(src + id), m);
                    mine[id] = e / zs * (a.dgates[row * k + j] - dot);
                }
        } else if (put_u) {
            for (int j = sub; j < k; j += L) {
                const unsigned id = ids[j];
                if (id < (unsigned)E) mine[id] = a.dgates[row * k + j];
            }
        }
        __syncwarp();
        float u[EPL];
#pragma unroll
        for (int i = 0; i < EPL; i += 4) {
            const float4 q = *reinterpret_cast<const float4*>(mine + expert<L>(i, sub));
            u[i] = q.x, u[i + 1] = q.y, u[i + 2] = q.z, u[i + 3] = q.w;
        }
        __syncwarp();
        if (put_u)
            for (int j = sub; j < k; j += L)
                if ((unsigned)ids[j] < (unsigned)E) mine[ids[j]] = 0.f;

        float z = 0.f, dot = 0.f;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            f[i] = exp_of(f[i], m);
            z += f[i];
            dot = fmaf(f[i], a.renorm ? ae[i] : ae[i] + u[i], dot);
        }
        z = group_sum<L>(z);
        dot = group_sum<L>(dot) / z;
        const float inv = 1.0f / z;
#pragma unroll
        for (int i = 0; i < EPL; i++) {
            const float p = f[i] * inv;
            f[i] = a.renorm ? fmaf(p, ae[i] - dot, u[i]) : p * (ae[i] + u[i] - dot);
            if (!valid) f[i] = 0.f;
        }
        if (on) store_row<T, L, R>((T*)a.dlogits + row * a.ldd, sub, E, a.vec, f);
        __syncwarp();
    }
    pdl_trigger();
}

// Blocks of the forward (rows of the partial sums) and of the backward: at
// most four an SM, each with two turns of its warps or more.
int64_t blocks_for(int64_t T, int64_t E) {
    int L = 1;
    while (L < 32 && L * 8 < E) L *= 2;
    const int64_t rows = (int64_t)NW * (32 / L) * 2;
    const int64_t b = (T + rows - 1) / rows;
    return b < 1 ? 1 : b > kDesignSMs * 4 ? kDesignSMs * 4 : b;
}

template <typename T, int L, int R>
cudaError_t run_fwd(const FwdArgs& a, int64_t P, cudaStream_t s) {
    return launch(router_fwd_kernel<T, L, R>, dim3((unsigned)P), dim3(NT), fwd_smem<L, R>(a.k), s,
                  true, a);
}
template <typename T, int L, int R>
cudaError_t run_bwd(const BwdArgs& a, int64_t P, cudaStream_t s) {
    return launch(router_bwd_kernel<T, L, R>, dim3((unsigned)P), dim3(NT), bwd_smem<L, R>(), s,
                  true, a);
}

// The lanes of a row follow from the number of experts alone.
#define ROUTER_BY_E(RUN, T)                             \
    (a.E <= 8     ? RUN<T, 1, 1>(a, P, s)               \
     : a.E <= 16  ? RUN<T, 2, 1>(a, P, s)               \
     : a.E <= 32  ? RUN<T, 4, 1>(a, P, s)               \
     : a.E <= 64  ? RUN<T, 8, 1>(a, P, s)               \
     : a.E <= 128 ? RUN<T, 16, 1>(a, P, s)              \
     : a.E <= 256 ? RUN<T, 32, 1>(a, P, s)              \
     : a.E <= 512 ? RUN<T, 32, 2>(a, P, s)              \
                  : RUN<T, 32, 4>(a, P, s))

bool vectors(const void* p, int64_t ld, int E, int es, int64_t T) {
    return E % 8 == 0 && (uintptr_t)p % 16 == 0 && (T <= 1 || ld * es % 16 == 0);
}

}  // namespace

int64_t router_tiles(int64_t T, int64_t E) { return T > 0 ? blocks_for(T, E) : 0; }

cudaError_t launch_router_fwd(const void* logits, int64_t ld, const unsigned char* mask, int64_t k,
                              int renorm, float* gates, int* ids, int* counts, float* loss,
                              void* workspace, int64_t T, int64_t E, int dtype, cudaStream_t s) {
    const int64_t P = router_tiles(T, E);
    float* part_p = (float*)workspace;
    int* part_c = (int*)(part_p + P * E);
    if (P > 0) {
        const FwdArgs a{logits, mask, gates, ids, part_p, part_c, ld, T, (int)E, (int)k, renorm,
                        vectors(logits, ld, (int)E, elt_bytes(dtype), T)};
        const cudaError_t e = dtype == 0   ? ROUTER_BY_E(run_fwd, float)
                              : dtype == 1 ? ROUTER_BY_E(run_fwd, __half)
                                           : ROUTER_BY_E(run_fwd, __nv_bfloat16);
        if (e != cudaSuccess) return e;
    }
    const unsigned cs = E <= 32 ? 1 : E <= 64 ? 2 : E <= 128 ? 4 : 8;
    return launch_cluster(router_reduce_kernel, 1, cs, dim3(RT), 0, s, (const float*)part_p,
                          (const int*)part_c, (int)P, (int)E, (int)k, counts, loss);
}

cudaError_t launch_router_bwd(const void* logits, int64_t ld, const int* ids, const int* counts,
                              int64_t k, int renorm, const float* dgates, const float* dloss,
                              void* dlogits, int64_t ldd, int64_t T, int64_t E, int dtype,
                              cudaStream_t s) {
    const int64_t P = router_tiles(T, E);
    if (P == 0) return cudaSuccess;
    const int es = elt_bytes(dtype);
    const BwdArgs a{logits, ids, counts, dgates, dloss, dlogits, ld, ldd, T, (int)E, (int)k, renorm,
                    vectors(logits, ld, (int)E, es, T) && vectors(dlogits, ldd, (int)E, es, T)};
    return dtype == 0   ? ROUTER_BY_E(run_bwd, float)
           : dtype == 1 ? ROUTER_BY_E(run_bwd, __half)
                        : ROUTER_BY_E(run_bwd, __nv_bfloat16);
}

}  // namespace wsf
