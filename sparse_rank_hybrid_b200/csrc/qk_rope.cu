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

constexpr size_t kRingBytes = 200 * 1024;  // dynamic shared memory of an SM's blocks at most

constexpr int rope_threads(int V) { return V == 1 ? 1024 : V == 2 ? 640 : 512; }

// Eight elements of a head: consecutive ones (interleaved pairs), or four of the lower half and the four
// they pair with in the upper half, `half` elements on.
template <typename T, bool HALVES>
__device__ __forceinline__ void copy_in(const Ring& ring, int u, const T* p, int half) {
    if constexpr (!HALVES) {
        ring.copy(u, p);
    } else if constexpr (sizeof(T) == 4) {
        async_copy16(ring.in + u * ring.unit, p);
        async_copy16(ring.in + (u + 1) * ring.unit, p + half);
    } else {
        async_copy8(ring.in + u * ring.unit, p);
        async_copy8(ring.in + u * ring.unit + 8, p + half);
    }
}
template <typename T, bool HALVES>
__device__ __forceinline__ void store_out(T* p, int half, const Vec& v) {
    uint4 u[kUnits<T>];
    pack<T>(v, u);
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
__device__ __forceinline__ float weight_at(const void* w, int dtype, int at) {
    return dtype == kF32    ? static_cast<const float*>(w)[at]
           : dtype == kBf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[at])
                            : __half2float(static_cast<const __half*>(w)[at]);
}

// The four pairs of a vector turned by their angles; the cos and sin of pairs (0, 1) and (2, 3) in c, s.
template <bool HALVES>
__device__ __forceinline__ void rotate(Vec& v, const float2 (&c)[2], const float2 (&s)[2]) {
    if constexpr (HALVES) {  // pairs m and m + 4: two pairs at once
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            const float2 lo = v.f[m], hi = v.f[m + 2], neg = make_float2(-s[m].x, -s[m].y);
            v.f[m] = fma2(hi, neg, mul2(lo, c[m]));
            v.f[m + 2] = fma2(hi, c[m], mul2(lo, s[m]));
        }
    } else {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            const float cc = m & 1 ? c[m / 2].y : c[m / 2].x, ss = m & 1 ? s[m / 2].y : s[m / 2].x;
            const float2 p = v.f[m];
            v.f[m] = make_float2(fmaf(-p.y, ss, p.x * cc), fmaf(p.y, cc, p.x * ss));
        }
    }
}

template <typename TX, typename TO, int V, bool HALVES, bool BWD, bool WIDE>
__global__ void __launch_bounds__(WIDE ? rope_threads(V) : 128) qk_rope_kernel(const __grid_constant__ QkRopeArgs a) {
    constexpr int UX = kUnits<TX>, UD = BWD ? kUnits<TO> : 0, ONE = UX + UD, U = V * ONE;
    using TW = typename std::conditional<BWD, TX, TO>::type;  // type of what is written
    extern __shared__ uint4 shared[];
    __shared__ __align__(16) float scratch[kTeamScratch];
    __shared__ double turns[kRopeMaxPairs];
    __shared__ int axis[kRopeMaxPairs];
    const int D = a.head_dim, pairs = D / 2, half = HALVES ? D / 2 : 0, G = a.group;
    const int team_size = WIDE ? blockDim.x : a.team;
    const int t = WIDE ? threadIdx.x : threadIdx.x % a.team, lane = t % G;
    const int in_block = WIDE ? 0 : threadIdx.x / a.team, teams = WIDE ? 1 : blockDim.x / a.team;
    const int worker = blockIdx.x * teams + in_block;
    const int q_heads = a.side[0].heads, heads = q_heads + a.side[1].heads;
    for (int j = threadIdx.x; j < pairs; j += blockDim.x) turns[j] = a.turns[j], axis[j] = a.axis[j];
    Team<WIDE> team(team_size, scratch);
    __syncthreads();
    // cos and sin of the current and the next token: [2][2][pairs] floats a team, behind the ring
    float* table = reinterpret_cast<float*>(shared + static_cast<size_t>(a.stages) * U * blockDim.x) + in_block * 4 * pairs;

    const long long r0 = worker_lo(a.rows, a.workers, worker), r1 = worker_lo(a.rows, a.workers, worker + 1);
    const int n = static_cast<int>(r1 - r0);
    const int iters = WIDE ? n : static_cast<int>((a.rows + a.workers - 1) / a.workers);
    const int b0 = static_cast<int>(r0 / a.tokens), l0 = static_cast<int>(r0 % a.tokens);
    const bool need_x = !BWD || a.norm != kQkNormNone;

    // this thread's vectors: which side and head, where, and whether there is one
    Ring ring(shared_address(shared), a.stages, U);
    const TX* px[V];
    const TO* pd[V];
    TW* po[V];
    Vec w[V], dw[V];
    bool is_k[V], on[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int head = (t + v * team_size) / G;
        on[v] = head < heads && lane * 8 < D;
        is_k[v] = head >= q_heads;
        const RopeSide& s = a.side[is_k[v]];
        const int h = on[v] ? head - (is_k[v] ? q_heads : 0) : 0, c = lane * (HALVES ? 4 : 8);
        px[v] = static_cast<const TX*>(s.x) + s.sx.row(b0, l0, h) + c;
        pd[v] = static_cast<const TO*>(s.d) + s.sd.row(b0, l0, h) + c;
        po[v] = static_cast<TW*>(s.out) + s.so.row(b0, l0, h) + c;
        if (!on[v]) ring.clear(v * ONE, ONE);
        w[v] = vec_of(1.f);
        dw[v] = vec_of(0.f);
        if (on[v] && a.norm && s.weight) {
            const int at = (a.norm == kQkNormToken ? h * D : 0) + c, up = at + (HALVES ? half : 4);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                w[v].f[e] = make_float2(weight_at(s.weight, a.w_dtype, at + 2 * e), weight_at(s.weight, a.w_dtype, at + 2 * e + 1));
                w[v].f[e + 2] = make_float2(weight_at(s.weight, a.w_dtype, up + 2 * e), weight_at(s.weight, a.w_dtype, up + 2 * e + 1));
            }
        }
    }

    int lp = l0, left = n;
    auto prefetch = [&]() {
        if (left > 0) {
            --left;
            const bool last = ++lp == a.tokens;
            if (last) lp = 0;
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const RopeSide& q = a.side[0];
                const RopeSide& k = a.side[1];
                if (need_x) {
                    if (on[v]) copy_in<TX, HALVES>(ring, v * ONE, px[v], half);
                    px[v] += is_k[v] ? k.sx.l : q.sx.l;
                    if (last) px[v] += is_k[v] ? k.sx.b - a.tokens * k.sx.l : q.sx.b - a.tokens * q.sx.l;
                }
                if (BWD) {
                    if (on[v]) copy_in<TO, HALVES>(ring, v * ONE + UX, pd[v], half);
                    pd[v] += is_k[v] ? k.sd.l : q.sd.l;
                    if (last) pd[v] += is_k[v] ? k.sd.b - a.tokens * k.sd.l : q.sd.b - a.tokens * q.sd.l;
                }
            }
            ring.filled();
        }
        async_commit();
    };
    for (int s = 0; s < a.stages - 1; ++s) prefetch();

    // The table of the row whose batch and token are (tb, tl), in half `which` of the team's table; its
    // grid place (gt, gh, gw) moves along with it.
    const long long start = a.first + l0;
    const int hw = a.positions ? 1 : a.H * a.W, gt0 = static_cast<int>(a.first / hw), g0 = static_cast<int>(a.first % hw);
    int tb = b0, tl = l0, gt = static_cast<int>(start / hw), gh = 0, gw = 0;
    if (!a.positions && a.rotate) gh = static_cast<int>(start % hw) / a.W, gw = static_cast<int>(start % hw) % a.W;
    auto fill = [&](int which) {
        float* cs = table + which * 2 * pairs;
        for (int j = t; j < pairs; j += team_size) {
            const int ax = axis[j];
            const int p = a.positions ? a.positions[tb * a.positions_b + tl * 3ll + ax] : ax == 0 ? gt : ax == 1 ? gh : gw;
            const double turn = static_cast<double>(p + a.offset[ax]) * turns[j];
            float sn, c;
            sincospif(2.0f * static_cast<float>(turn - rint(turn)), &sn, &c);
            cs[j] = c;
            cs[pairs + j] = BWD ? -sn : sn;  // the gradient turns back
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
    const float inv_q = 1.0f / (static_cast<float>(D) * q_heads);
    const float inv_k = 1.0f / (static_cast<float>(D) * max(1, a.side[1].heads));
    const bool has_pairs = lane * 8 < D;
    int l = l0;
    for (int i = 0; i < iters; ++i) {
        prefetch();
        const bool row = WIDE || i < n;
        float2 c[2] = {both(1.f), both(1.f)}, sn[2] = {both(0.f), both(0.f)};
        if (a.rotate) {
            if (has_pairs) {
                const float4* cs = reinterpret_cast<const float4*>(table + (i & 1) * 2 * pairs);
                const float4 u = cs[lane], z = cs[pairs / 4 + lane];
                c[0] = make_float2(u.x, u.y), c[1] = make_float2(u.z, u.w);
                sn[0] = make_float2(z.x, z.y), sn[1] = make_float2(z.z, z.w);
            }
            if (i + 1 < n) fill((i + 1) & 1);
            // every thread has read this row's table and sees the next one after a barrier of the team
            if (!WIDE || a.norm != kQkNormToken) team.sync();
        }
        ring_wait(a.stages);

        Vec x[V], g[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (need_x) x[v] = ring.read<TX>(v * ONE);
            if (BWD) {
                g[v] = ring.read<TO>(v * ONE + UX);
                if (a.rotate) rotate<HALVES>(g[v], c, sn);
            }
        }
        ring.done();
        // per vector: r, and r^2 mean(g w x) of the norm it belongs to
        float r[V], gx[V];
        if (a.norm) {
            float qq[V], z[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float2 s1 = mul2(x[v].f[0], x[v].f[0]), s2 = both(0.f);
#pragma unroll
                for (int e = 1; e < 4; ++e) s1 = fma2(x[v].f[e], x[v].f[e], s1);
                if (BWD)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s2 = fma2(mul2(g[v].f[e], w[v].f[e]), x[v].f[e], s2);
                qq[v] = fold(s1);
                z[v] = BWD ? fold(s2) : 0.f;
            }
            if (a.norm == kQkNormHead) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    for (int o = G >> 1; o > 0; o >>= 1) {
                        qq[v] += Team<WIDE>::swap(qq[v], o);
                        if (BWD) z[v] += Team<WIDE>::swap(z[v], o);
                    }
                    r[v] = rsqrtf(qq[v] * inv_head + a.eps);
                    if (BWD) gx[v] = z[v] * inv_head * r[v] * r[v];
                }
            } else {
                float q[BWD ? 4 : 2] = {};
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    q[0] += is_k[v] ? 0.f : qq[v];
                    q[1] += is_k[v] ? qq[v] : 0.f;
                    if constexpr (BWD) {
                        q[2] += is_k[v] ? 0.f : z[v];
                        q[3] += is_k[v] ? z[v] : 0.f;
                    }
                }
                team.sum(q);
                const float rq = rsqrtf(q[0] * inv_q + a.eps), rk = rsqrtf(q[1] * inv_k + a.eps);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    r[v] = is_k[v] ? rk : rq;
                    if constexpr (BWD) gx[v] = is_k[v] ? q[3] * inv_k * rk * rk : q[2] * inv_q * rq * rq;
                }
            }
        }
        const bool last = l + 1 == a.tokens;
        l = last ? 0 : l + 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            if (!BWD) {
                if (a.norm)
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[v].f[e] = mul2(x[v].f[e], mul2(w[v].f[e], both(r[v])));
                if (a.rotate) rotate<HALVES>(x[v], c, sn);
                if (row && on[v]) store_out<TW, HALVES>(po[v], half, x[v]);
            } else {
                if (a.norm) {
                    const float2 rr = both(r[v]), mg = both(-gx[v]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        if (row) dw[v].f[e] = fma2(g[v].f[e], mul2(x[v].f[e], rr), dw[v].f[e]);
                        g[v].f[e] = mul2(rr, fma2(x[v].f[e], mg, mul2(g[v].f[e], w[v].f[e])));
                    }
                }
                if (row && on[v]) store_out<TW, HALVES>(po[v], half, g[v]);
            }
            const Strides& sq = a.side[0].so;
            const Strides& sk = a.side[1].so;
            po[v] += is_k[v] ? sk.l : sq.l;
            if (last) po[v] += is_k[v] ? sk.b - a.tokens * sk.l : sq.b - a.tokens * sq.l;
        }
    }

    if (!BWD || !a.part) return;
    if (a.norm == kQkNormToken) {
        float* part = a.part + static_cast<long long>(worker) * heads * D;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (on[v]) store_out<float, HALVES>(part + (t + v * team_size) / G * D + lane * (HALVES ? 4 : 8), half, dw[v]);
        return;
    }
    // one weight for all heads of a side: joined over the heads in order, through the ring's memory
    async_wait<0>();
    __syncthreads();
    Vec* sums = reinterpret_cast<Vec*>(shared);
#pragma unroll
    for (int v = 0; v < V; ++v) sums[v * blockDim.x + threadIdx.x] = dw[v];
    __syncthreads();
    const int sides = heads > q_heads ? 2 : 1;
    for (int j = t; j < sides * G; j += team_size) {
        const int side = j / G, place = j % G;
        if (place * 8 >= D) continue;
        Vec d = vec_of(0.f);
        for (int h = side ? q_heads : 0; h < (side ? heads : q_heads); ++h) {
            const int slot = h * G + place, v = slot / team_size, at = in_block * team_size + slot % team_size;
            const Vec u = sums[v * blockDim.x + at];
#pragma unroll
            for (int e = 0; e < 4; ++e) d.f[e] = add2(d.f[e], u.f[e]);
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

// Blocks that a processor holds at once, from the registers the kernels need.
int blocks_per_sm(const RowPlan& p, bool backward) { return std::max(1, (p.V == 1 ? 1024 : 640) / p.threads); }

template <typename TX, typename TO, int V, bool HALVES, bool BWD, bool WIDE>
cudaError_t launch(QkRopeArgs a, const RowPlan& p, cudaStream_t st) {
    const size_t stage = size_t(16) * V * (kUnits<TX> + (BWD ? kUnits<TO> : 0)) * p.threads;
    const int per_sm = blocks_per_sm(p, BWD);
    a.stages = ring_stages(stage, per_sm, kRingBytes / per_sm);
    const size_t smem = a.stages * stage + size_t(p.threads / p.team) * 2 * a.head_dim * sizeof(float);
    const auto kernel = qk_rope_kernel<TX, TO, V, HALVES, BWD, WIDE>;
    if (smem > 40 * 1024) {  // 48 KB without opting in, less the static part
        const cudaError_t e =
            cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
    }
    kernel<<<p.blocks, p.threads, smem, st>>>(a);
    return cudaGetLastError();
}
template <typename TX, typename TO, int V, bool WIDE>
cudaError_t launch_dir(const QkRopeArgs& a, const RowPlan& p, bool backward, cudaStream_t st) {
    if (a.halves)
        return backward ? launch<TX, TO, V, true, true, WIDE>(a, p, st) : launch<TX, TO, V, true, false, WIDE>(a, p, st);
    return backward ? launch<TX, TO, V, false, true, WIDE>(a, p, st) : launch<TX, TO, V, false, false, WIDE>(a, p, st);
}
template <typename TX, typename TO>
cudaError_t launch_types(const QkRopeArgs& a, const RowPlan& p, bool backward, cudaStream_t st) {
    return p.team <= 32 ? launch_dir<TX, TO, 1, false>(a, p, backward, st)
           : p.V == 1   ? launch_dir<TX, TO, 1, true>(a, p, backward, st)
           : p.V == 2   ? launch_dir<TX, TO, 2, true>(a, p, backward, st)
                        : launch_dir<TX, TO, 4, true>(a, p, backward, st);
}

}  // namespace

RowPlan qk_rope_plan(long long rows, int head_dim, int heads, bool backward) {
    RowPlan p;
    const int slots = heads * group_of(head_dim);
    int V = 1;
    while (V < 4 && (slots + V - 1) / V > rope_threads(V)) V *= 2;
    row_team(slots, V, &p);
    row_workers(rows, kSMs * blocks_per_sm(p, backward), &p);
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
