// QK norm and rotary positions along (t, h, w) in one pass over the tokens, and its gradient.
//
//   forward   n = x r, r = rsqrt(mean(x^2) + e), the mean over a head's D elements or over all heads of
//             the token (or n = x);  out = R(p) (n w), each pair (a, b) of a head turned by
//             p[axis_j] omega_j: (a c - b s, a s + b c)
//   backward  g = R(p)^T dout, dw = sum g n, dx = r (g w - n mean(g w n)); both means need only
//             sum(x^2) and sum(g w x), one joint sum over the row
//
// Bound by memory.  A team of threads takes all heads of a token's q and k together: thread and vector
// of eight elements have a fixed (head, place in the head) for every token, so the weights and the
// gradient sums of the weights stay in registers, and the token's angles are computed once for all heads.
// The angle is a product in double (turns = omega / 2 pi per position), of which only the fraction of a
// turn goes on to fp32: positions of any size keep an error below 1e-7 of a turn.  The table of a token's
// cos and sin is filled while the token before it is computed.  Rows travel through a per-thread ring of
// asynchronous copies as in residual_norm.cu.
#include <algorithm>
#include <type_traits>

#include "rows.cuh"

namespace slra {
namespace {

constexpr int kMaxStages = 3;
constexpr size_t kRingBytes = 200 * 1024;  // of a block's dynamic shared memory at most

constexpr int rope_threads(int V) { return V == 1 ? 1024 : V == 2 ? 640 : 512; }

// Eight elements of a head: consecutive ones (interleaved pairs), or four of the lower half and the four
// they pair with in the upper half, `half` elements on.
template <typename T, bool HALVES>
__device__ __forceinline__ void copy_in(uint4* s, int step, const T* p, int half) {
    if constexpr (!HALVES) {
#pragma unroll
        for (int i = 0; i < kUnits<T>; ++i) async_copy16(s + i * step, reinterpret_cast<const uint4*>(p) + i);
    } else if constexpr (sizeof(T) == 4) {
        async_copy16(s, p);
        async_copy16(s + step, p + half);
    } else {
        async_copy8(s, p);
        async_copy8(reinterpret_cast<uint2*>(s) + 1, p + half);
    }
}
template <typename T, bool HALVES>
__device__ __forceinline__ void store_out(T* p, int half, const float (&f)[8]) {
    uint4 u[kUnits<T>];
    pack8<T>(f, u);
    if constexpr (!HALVES) {
#pragma unroll
        for (int i = 0; i < kUnits<T>; ++i) reinterpret_cast<uint4*>(p)[i] = u[i];
    } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<uint4*>(p) = u[0];
        *reinterpret_cast<uint4*>(p + half) = u[1];
    } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(u[0].x, u[0].y);
        *reinterpret_cast<uint2*>(p + half) = make_uint2(u[0].z, u[0].w);
    }
}
template <bool HALVES>
__device__ __forceinline__ float weight_at(const void* w, int dtype, int at, int half, int e) {
    if (!w) return 1.f;
    const int i = at + e + (HALVES && e >= 4 ? half - 4 : 0);
    return dtype == kF32    ? static_cast<const float*>(w)[i]
           : dtype == kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i])
                            : __half2float(static_cast<const __half*>(w)[i]);
}

template <bool HALVES>
__device__ __forceinline__ void rotate(float (&f)[8], const float (&c)[4], const float (&s)[4], float sign) {
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        const int i = HALVES ? m : 2 * m, j = HALVES ? m + 4 : 2 * m + 1;
        const float a = f[i], b = f[j], sn = sign * s[m];
        f[i] = a * c[m] - b * sn;
        f[j] = a * sn + b * c[m];
    }
}

template <typename TX, typename TO, int V, bool HALVES, bool BWD>
__global__ void __launch_bounds__(rope_threads(V)) qk_rope_kernel(const __grid_constant__ QkRopeArgs a) {
    constexpr int UX = kUnits<TX>, UD = BWD ? kUnits<TO> : 0, U = V * (UX + UD);
    using TW = typename std::conditional<BWD, TX, TO>::type;  // type of what is written
    extern __shared__ uint4 ring[];
    __shared__ float scratch[kTeamScratch];
    __shared__ double turns[kRopeMaxPairs];
    __shared__ int axis[kRopeMaxPairs];
    const int D = a.head_dim, pairs = D / 2, half = HALVES ? D / 2 : 0, G = a.group;
    const int t = threadIdx.x % a.team, lane = t % G, in_block = threadIdx.x / a.team;
    const int teams = blockDim.x / a.team, worker = blockIdx.x * teams + in_block;
    const int heads = a.side[0].heads + a.side[1].heads;
    Team team{a.team, scratch, 0};
    // cos and sin of the current and the next token: [2][2][pairs] floats a team, behind the ring
    float* table = reinterpret_cast<float*>(ring + static_cast<size_t>(a.stages) * U * blockDim.x) + in_block * 4 * pairs;
    for (int j = threadIdx.x; j < pairs; j += blockDim.x) turns[j] = a.turns[j], axis[j] = a.axis[j];
    __syncthreads();

    const long long r0 = worker_lo(a.rows, a.workers, worker), r1 = worker_lo(a.rows, a.workers, worker + 1);
    const int n = static_cast<int>(r1 - r0);
    const int iters = a.team <= 32 ? static_cast<int>((a.rows + a.workers - 1) / a.workers) : n;
    const int b0 = static_cast<int>(r0 / a.tokens), l0 = static_cast<int>(r0 % a.tokens);
    const bool need_x = !BWD || a.norm != kQkNormNone;

    // this thread's vectors: which side and head, where, and whether there is one
    const TX* px[V];
    const TO* pd[V];
    TW* po[V];
    float w[V][8], dw[V][8];
    bool is_k[V], live[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int head = (t + v * a.team) / G;
        live[v] = head < heads && lane * 8 < D;
        is_k[v] = head >= a.side[0].heads;
        const RopeSide& s = a.side[is_k[v]];
        const int h = live[v] ? head - (is_k[v] ? a.side[0].heads : 0) : 0, c = lane * (HALVES ? 4 : 8);
        px[v] = static_cast<const TX*>(s.x) + s.sx.row(b0, l0, h) + c;
        pd[v] = static_cast<const TO*>(s.d) + s.sd.row(b0, l0, h) + c;
        po[v] = static_cast<TW*>(s.out) + s.so.row(b0, l0, h) + c;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            w[v][e] = live[v] && a.norm ? weight_at<HALVES>(s.weight, a.w_dtype, (a.norm == kQkNormToken ? h * D : 0) + c, half, e) : 1.f;
            dw[v][e] = 0.f;
        }
    }

    int lp = l0, left = n;
    auto prefetch = [&](int stage) {
        if (left > 0) {
            --left;
            uint4* s = ring + static_cast<size_t>(stage) * U * blockDim.x + threadIdx.x;
            const bool last = ++lp == a.tokens;
            if (last) lp = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!live[v]) continue;
                const RopeSide& side = a.side[is_k[v]];
                if (need_x) {
                    copy_in<TX, HALVES>(s + v * UX * blockDim.x, blockDim.x, px[v], half);
                    px[v] += last ? side.sx.b - (a.tokens - 1) * side.sx.l : side.sx.l;
                }
                if (BWD) {
                    copy_in<TO, HALVES>(s + (V * UX + v * UD) * blockDim.x, blockDim.x, pd[v], half);
                    pd[v] += last ? side.sd.b - (a.tokens - 1) * side.sd.l : side.sd.l;
                }
            }
        }
        async_commit();
    };
    for (int s = 0; s < a.stages - 1; ++s) prefetch(s);

    // The table of the row whose batch and token are (tb, tl), in half `which` of the team's table; its
    // grid place (gt, gh, gw) moves along with it.
    const long long start = a.first + l0;
    const int hw = a.positions ? 1 : a.H * a.W, gt0 = static_cast<int>(a.first / hw), g0 = static_cast<int>(a.first % hw);
    int tb = b0, tl = l0, gt = static_cast<int>(start / hw), gh = 0, gw = 0;
    if (!a.positions && a.rotate) gh = static_cast<int>(start % hw) / a.W, gw = static_cast<int>(start % hw) % a.W;
    auto fill = [&](int which) {
        float* cs = table + which * 2 * pairs;
        for (int j = t; j < pairs; j += a.team) {
            const int ax = axis[j];
            const int p = a.positions ? a.positions[tb * a.positions_b + tl * 3ll + ax] : ax == 0 ? gt : ax == 1 ? gh : gw;
            const double turn = static_cast<double>(p + a.offset[ax]) * turns[j];
            float sn, c;
            sincospif(2.0f * static_cast<float>(turn - rint(turn)), &sn, &c);
            cs[j] = c;
            cs[pairs + j] = sn;
        }
        if (++tl == a.tokens) {
            tl = 0, ++tb;
            if (!a.positions) gt = gt0, gh = g0 / a.W, gw = g0 % a.W;
        } else if (++gw == a.W) {
            gw = 0;
            if (++gh == a.H) gh = 0, ++gt;
        }
    };
    if (a.rotate) {
        if (n > 0) fill(0);
        team.sync();
    }

    const float inv_head = 1.0f / D;
    const float inv_q = 1.0f / (static_cast<float>(D) * a.side[0].heads);
    const float inv_k = 1.0f / (static_cast<float>(D) * max(1, a.side[1].heads));
    int stage = 0, l = l0;
    for (int i = 0; i < iters; ++i) {
        prefetch(stage == 0 ? a.stages - 1 : stage - 1);
        const bool row = i < n;
        float c[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
        if (a.rotate) {
            if (row && lane * 8 < D) {
                const float4* cs = reinterpret_cast<const float4*>(table + (i & 1) * 2 * pairs);
                const float4 u = cs[lane], z = cs[pairs / 4 + lane];
                c[0] = u.x, c[1] = u.y, c[2] = u.z, c[3] = u.w;
                sn[0] = z.x, sn[1] = z.y, sn[2] = z.z, sn[3] = z.w;
            }
            if (i + 1 < n) fill((i + 1) & 1);
            // every thread has read this row's table and sees the next one after a barrier of the team
            if (a.norm != kQkNormToken || a.team <= 32) team.sync();
        }
        if (a.stages == 3) async_wait<2>();
        else if (a.stages == 2) async_wait<1>();
        else async_wait<0>();
        const uint4* s = ring + static_cast<size_t>(stage) * U * blockDim.x + threadIdx.x;
        if (++stage == a.stages) stage = 0;

        float x[V][8], g[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const bool on = row && live[v];
            if (on && need_x) {
                uint4 u[UX];
#pragma unroll
                for (int k = 0; k < UX; ++k) u[k] = s[(v * UX + k) * blockDim.x];
                unpack8<TX>(u, x[v]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[v][e] = 0.f;
            }
            if (BWD) {
                if (on) {
                    uint4 u[kUnits<TO>];
#pragma unroll
                    for (int k = 0; k < UD; ++k) u[k] = s[(V * UX + v * UD + k) * blockDim.x];
                    unpack8<TO>(u, g[v]);
                    rotate<HALVES>(g[v], c, sn, -1.f);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) g[v][e] = 0.f;
                }
            }
        }
        // per vector: r, and r^2 mean(g w x) of the norm it belongs to
        float r[V], gx[V];
        if (a.norm == kQkNormHead) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float q = 0.f, z = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    q += x[v][e] * x[v][e];
                    if (BWD) z += g[v][e] * w[v][e] * x[v][e];
                }
                for (int o = G >> 1; o > 0; o >>= 1) {
                    q += __shfl_xor_sync(0xffffffffu, q, o);
                    if (BWD) z += __shfl_xor_sync(0xffffffffu, z, o);
                }
                r[v] = rsqrtf(q * inv_head + a.eps);
                gx[v] = z * inv_head * r[v] * r[v];
            }
        } else if (a.norm == kQkNormToken) {
            float q[BWD ? 4 : 2] = {};
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float qq = 0.f, z = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    qq += x[v][e] * x[v][e];
                    if (BWD) z += g[v][e] * w[v][e] * x[v][e];
                }
                q[0] += is_k[v] ? 0.f : qq;
                q[1] += is_k[v] ? qq : 0.f;
                if (BWD) {
                    q[BWD ? 2 : 0] += is_k[v] ? 0.f : z;
                    q[BWD ? 3 : 0] += is_k[v] ? z : 0.f;
                }
            }
            team.sum(q);
            const float rq = rsqrtf(q[0] * inv_q + a.eps), rk = rsqrtf(q[1] * inv_k + a.eps);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                r[v] = is_k[v] ? rk : rq;
                if (BWD) gx[v] = is_k[v] ? q[BWD ? 3 : 0] * inv_k * rk * rk : q[BWD ? 2 : 0] * inv_q * rq * rq;
            }
        }
        if (row) {
            const bool last = ++l == a.tokens;
            if (last) l = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (!live[v]) continue;
                const RopeSide& side = a.side[is_k[v]];
                if (!BWD) {
                    if (a.norm)
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[v][e] = x[v][e] * r[v] * w[v][e];
                    rotate<HALVES>(x[v], c, sn, 1.f);
                    store_out<TW, HALVES>(po[v], half, x[v]);
                } else {
                    if (a.norm)
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            dw[v][e] = fmaf(g[v][e], x[v][e] * r[v], dw[v][e]);
                            g[v][e] = r[v] * (g[v][e] * w[v][e] - x[v][e] * gx[v]);
                        }
                    store_out<TW, HALVES>(po[v], half, g[v]);
                }
                po[v] += last ? side.so.b - (a.tokens - 1) * side.so.l : side.so.l;
            }
        }
    }

    if (!BWD || !a.part) return;
    if (a.norm == kQkNormToken) {
        float* part = a.part + static_cast<long long>(worker) * heads * D;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (live[v]) store_out<float, HALVES>(part + (t + v * a.team) / G * D + lane * (HALVES ? 4 : 8), half, dw[v]);
        return;
    }
    // one weight for all heads of a side: joined over the heads in order, through the ring's memory
    async_wait<0>();
    __syncthreads();
    float4* sums = reinterpret_cast<float4*>(ring);
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int k = 0; k < 2; ++k)
            sums[(v * 2 + k) * blockDim.x + threadIdx.x] =
                make_float4(dw[v][4 * k], dw[v][4 * k + 1], dw[v][4 * k + 2], dw[v][4 * k + 3]);
    __syncthreads();
    const int sides = a.side[1].heads > 0 ? 2 : 1;
    for (int j = t; j < sides * G; j += a.team) {
        const int side = j / G, place = j % G;
        if (place * 8 >= D) continue;
        const int h0 = side ? a.side[0].heads : 0, h1 = side ? heads : a.side[0].heads;
        float d[8] = {};
        for (int h = h0; h < h1; ++h) {
            const int slot = h * G + place, v = slot / a.team, at = in_block * a.team + slot % a.team;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float4 u = sums[(v * 2 + k) * blockDim.x + at];
                d[4 * k] += u.x, d[4 * k + 1] += u.y, d[4 * k + 2] += u.z, d[4 * k + 3] += u.w;
            }
        }
        store_out<float, HALVES>(a.part + (static_cast<long long>(worker) * sides + side) * D + place * (HALVES ? 4 : 8),
                                 half, d);
    }
}

// The weights' gradients: the workers' sums joined in a fixed order, 32 columns a block.
constexpr int kFinalWarps = 16;
__global__ void __launch_bounds__(32 * kFinalWarps) qk_rope_final_kernel(const float* part, int workers, int columns,
                                                                         int q_columns, float* dwq, float* dwk) {
    __shared__ float red[kFinalWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (c < columns)
        for (int w = warp; w < workers; w += kFinalWarps) sum += part[static_cast<long long>(w) * columns + c];
    red[warp][lane] = sum;
    __syncthreads();
    if (warp != 0 || c >= columns) return;
    sum = 0.f;
    for (int w = 0; w < kFinalWarps; ++w) sum += red[w][lane];
    if (c < q_columns) {
        if (dwq) dwq[c] = sum;
    } else if (dwk) {
        dwk[c - q_columns] = sum;
    }
}

int group_of(int head_dim) {
    int g = 1;
    while (g * 8 < head_dim) g *= 2;
    return g;
}

template <typename TX, typename TO, int V, bool HALVES, bool BWD>
cudaError_t launch(QkRopeArgs a, const RowPlan& p, cudaStream_t st) {
    const size_t stage = size_t(16) * V * (kUnits<TX> + (BWD ? kUnits<TO> : 0)) * p.threads;
    a.stages = kMaxStages;
    while (a.stages > 1 && a.stages * stage > kRingBytes) --a.stages;
    const size_t smem = a.stages * stage + size_t(p.threads / p.team) * 2 * a.head_dim * sizeof(float);
    const auto kernel = qk_rope_kernel<TX, TO, V, HALVES, BWD>;
    if (smem > 40 * 1024) {  // 48 KB without opting in, less the static part
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    kernel<<<p.blocks, p.threads, smem, st>>>(a);
    return cudaGetLastError();
}
template <typename TX, typename TO, int V>
cudaError_t launch_dir(const QkRopeArgs& a, const RowPlan& p, bool backward, cudaStream_t st) {
    if (a.halves)
        return backward ? launch<TX, TO, V, true, true>(a, p, st) : launch<TX, TO, V, true, false>(a, p, st);
    return backward ? launch<TX, TO, V, false, true>(a, p, st) : launch<TX, TO, V, false, false>(a, p, st);
}
template <typename TX, typename TO>
cudaError_t launch_types(const QkRopeArgs& a, const RowPlan& p, bool backward, cudaStream_t st) {
    return p.V == 1   ? launch_dir<TX, TO, 1>(a, p, backward, st)
           : p.V == 2 ? launch_dir<TX, TO, 2>(a, p, backward, st)
                      : launch_dir<TX, TO, 4>(a, p, backward, st);
}

}  // namespace

RowPlan qk_rope_plan(long long rows, int head_dim, int heads, bool backward) {
    RowPlan p;
    const int G = group_of(head_dim), slots = heads * G;
    p.V = 1;
    if (slots <= 32) {
        p.team = 1;
        while (p.team < slots) p.team *= 2;
        p.threads = 128;
    } else {
        while (p.V < 4 && (slots + p.V - 1) / p.V > rope_threads(p.V)) p.V *= 2;
        p.team = p.threads = ((slots + p.V - 1) / p.V + 31) / 32 * 32;
    }
    const int teams = p.threads / p.team;
    const int per_sm = std::max(1, (backward ? 640 : 1024) / p.threads);
    const long long want = (rows + teams - 1) / teams;
    p.blocks = static_cast<int>(std::min<long long>(want, std::min(kSMs * per_sm, kMaxWorkers / teams)));
    p.workers = p.blocks * teams;
    return p;
}

cudaError_t launch_qk_rope(const QkRopeArgs& args, bool backward, cudaStream_t st) {
    QkRopeArgs a = args;
    const int heads = a.side[0].heads + a.side[1].heads;
    const RowPlan p = qk_rope_plan(a.rows, a.head_dim, heads, backward);
    a.group = group_of(a.head_dim);
    a.team = p.team;
    a.workers = p.workers;
    cudaError_t e;
    if (a.x_dtype == kF32)
        e = launch_types<float, float>(a, p, backward, st);
    else if (a.x_dtype == kBf16)
        e = a.out_dtype == kF32 ? launch_types<__nv_bfloat16, float>(a, p, backward, st)
                                : launch_types<__nv_bfloat16, __nv_bfloat16>(a, p, backward, st);
    else
        e = a.out_dtype == kF32 ? launch_types<__half, float>(a, p, backward, st)
                                : launch_types<__half, __half>(a, p, backward, st);
    if (e != cudaSuccess || !backward || !a.part) return e;
    const bool per_head = a.norm == kQkNormToken;  // a weight for each head
    const int q_columns = a.head_dim * (per_head ? a.side[0].heads : 1);
    const int k_columns = a.head_dim * (per_head ? a.side[1].heads : a.side[1].heads > 0);
    const int columns = q_columns + k_columns;
    qk_rope_final_kernel<<<(columns + 31) / 32, 32 * kFinalWarps, 0, st>>>(a.part, p.workers, columns, q_columns,
                                                                           a.side[0].dweight, a.side[1].dweight);
    return cudaGetLastError();
}

}  // namespace slra
