// QK norm and rotary positions along (t, h, w) in one pass over the tokens, and its gradient.
//
//   forward   n = x r, r = rsqrt(mean(x^2) + e), the mean over a head's D elements or over all heads of
//             the token (or n = x);  out = R(p) (n w), each pair (a, b) of a head turned by
//             p[axis_j] omega_j: (a c - b s, a s + b c)
//   backward  g = R(p)^T dout, dw = sum g n, dx = r (g w - n mean(g w n)); both means need only
//             sum(x^2) and sum(g w x), one joint sum over the row
//
// Bound by memory.  A team of threads takes all heads of a token (or a part of them, or q's or k's alone: see
// the plan in qk_rope.cu): thread and vector of eight elements have a fixed head and place in it for every
// token, so the weights and their gradients' sums stay in registers, and a token's angles are computed once
// for all heads.  The angle is counted in turns as an integer: position times omega / 2 pi in units of 2^-64
// of a turn wraps around at whole turns by itself, so its upper half is the fraction of a turn to 2^-32
// wherever the position is, for three integer multiplications (a double product with its rounding to a whole
// number took most of the time of a step).  The table of a step's cos and sin is filled during the step
// before it.  Pairs that are not rotated pass through as they are: a product with (1, 0) would make NaN of an
// infinity's partner and lose the sign of zeros.  Rows travel through a per-thread ring of asynchronous copies
// (rows.cuh).
//
// B200, back to back, against 6557 GB/s of copy rate, over cards and places of the buffers: 75,600 tokens x 2 x
// 40 heads of 128, bf16, norm per head: forward 0.47-0.54 ms (87-99%), backward 0.86-0.94 ms (75-82%); 32,760 x
// 2 x 12 heads, norm over the heads: forward out of a fused projection 76-79 us (78-81%), backward from fp32
// gradients 146-159 us (77-84%); the same norms without the rotation 0.47-0.51 and 0.83-0.87 ms, 72-76 and
// 137-140 us.  What keeps the backward and the short rows from the rate is issue: 202 to 246 instructions a
// warp and vector in the backward, 110 to 129 in the forward.
#pragma once

#include <algorithm>
#include <type_traits>

#include "rows.cuh"

namespace slra {

constexpr size_t kRopeRingBytes = 200 * 1024;  // dynamic shared memory of the rings of an SM's blocks at most
// and of a block's tables: two steps of two tokens for each team, whose heads have 256 elements, or 1024 together
// where teams share a block
constexpr size_t kRopeTableBytes = 2 * 2 * 1024 * sizeof(float);

// Tokens that a team takes at a time, for V vectors a thread: what a step costs besides its vectors (the
// loop, the ring, the table, the barrier and the sums' exchanges) is shared by them, while the weights and
// their gradients' sums stay in the same registers (720p forward with one: 641 us, with two 492).  The
// backward has registers for two vectors in all.
template <int V, bool BWD>
constexpr int kRows = BWD && V > 1 ? 1 : 2;

// Threads of a block at most, so that the registers hold V vectors of kRows tokens with their weights and,
// in the backward, the weights' sums.
constexpr int rope_threads(int V, bool backward) {
    return V == 1 ? 640 : V == 2 ? (backward ? 512 : 640) : (backward ? 320 : 512);
}
// Blocks of that many threads (narrow: of 128) that an SM has to hold.  The backward without a norm, a rotation
// alone, needs 48 to 64 registers a thread; with the choice of rotate_some the compiler would take up to 82 (0: as it
// sees fit).
constexpr int rope_blocks(int V, bool wide, bool choice) { return !choice ? 0 : !wide ? 8 : V == 3 ? 3 : 2; }

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

// The cosine that the tables hold for a pair that is not rotated.
constexpr float kUnrotated = 2.f;

// As `rotate`, where some of the calls' pairs are not rotated.
template <bool HALVES>
__device__ __forceinline__ void rotate_some(Vec& v, const float2 (&c)[2], const float2 (&s)[2]) {
    const Vec u = v;
    rotate<HALVES>(v, c, s);
#pragma unroll
    for (int m = 0; m < 4; ++m) {  // the pair's cosine and its two elements
        const float cc = m & 1 ? c[m / 2].y : c[m / 2].x;
        if (cc != kUnrotated) continue;
        if constexpr (HALVES) {
            if (m & 1) v.f[m / 2].y = u.f[m / 2].y, v.f[m / 2 + 2].y = u.f[m / 2 + 2].y;
            else v.f[m / 2].x = u.f[m / 2].x, v.f[m / 2 + 2].x = u.f[m / 2 + 2].x;
        } else {
            v.f[m] = u.f[m];
        }
    }
}

// A vector is eight consecutive elements of a head, or four of each half (SPLIT): where the halves are paired,
// and where a tensor is fp32, so that a warp's accesses cover consecutive memory (480p backward from fp32
// gradients: 197 -> 146 us).  Of a thread's vectors VQ are of q and VK of k; without the latter they are of
// the side that the block takes.
template <typename TX, typename TO, int VQ, int VK, bool HALVES, bool BWD, bool WIDE, int NORM, bool ALL>
__global__ void __launch_bounds__(WIDE ? rope_threads(VQ + VK, BWD) : 128,
                                  rope_blocks(VQ + VK, WIDE, BWD && NORM == kQkNormNone && !ALL))
    qk_rope_kernel(const __grid_constant__ QkRopeArgs a) {
    // ALL: every pair is rotated.  Compiled apart: the choice at run time costs those calls up to 3%.
    // The backward is compiled for each norm: it issues so many instructions that the choice at run time
    // costs it a fifth (720p, norm per head: 1014 -> 861 us); the forward does not notice.
    const int norm = NORM < 0 ? a.norm : NORM;
    constexpr int V = VQ + VK, R = kRows<V, BWD>;
    constexpr int UX = kUnits<TX>, UD = BWD ? kUnits<TO> : 0, ONE = UX + UD, U = R * V * ONE;
    using TW = typename std::conditional<BWD, TX, TO>::type;  // type of what is written
    constexpr bool SPLIT = HALVES || sizeof(TX) == 4 || sizeof(TO) == 4;
    extern __shared__ uint4 shared[];
    __shared__ __align__(16) float scratch[kTeamScratch];
    __shared__ unsigned long long turns[kRopeMaxPairs];
    __shared__ int axis[kRopeMaxPairs];
    const int D = a.head_dim, pairs = D / 2, gap = SPLIT ? D / 2 : 4, G = a.group;
    const int team_size = WIDE ? blockDim.x : a.team;
    const int t = WIDE ? threadIdx.x : threadIdx.x % a.team, lane = t % G, c0 = lane * (SPLIT ? 4 : 8);
    const int in_block = WIDE ? 0 : threadIdx.x / a.team, teams = WIDE ? 1 : blockDim.x / a.team;
    const int part = blockIdx.x % a.parts, worker = blockIdx.x / a.parts * teams + in_block;
    for (int j = threadIdx.x; j < pairs; j += blockDim.x) turns[j] = a.turns[j], axis[j] = a.axis[j];
    Team<WIDE> team(team_size, scratch);
    __syncthreads();
    // cos and sin of this step's and the next one's tokens: [2][R][2][pairs] floats a team, behind the ring
    float* table = reinterpret_cast<float*>(shared + static_cast<size_t>(a.stages) * U * blockDim.x) + in_block * 4 * R * pairs;

    const long long r0 = static_cast<long long>(worker) * a.share;
    const int n = static_cast<int>(min(static_cast<long long>(a.share), max(0ll, a.rows - r0)));
    // teams of one warp take part in each other's shuffles, so they all loop as long as the longest
    const int longest = WIDE ? n : a.share;
    const int b0 = static_cast<int>(r0 / a.tokens), l0 = static_cast<int>(r0 % a.tokens);
    const bool need_x = !BWD || norm != kQkNormNone;

    // this block's heads of each side, and this thread's vectors: the head, and where it is in a token
    const int piece = a.split_sides ? 0 : part, side_q = VK == 0 && a.split_sides ? part : 0;
    Ring ring(shared_address(shared), a.stages, U);
    int head[V];
    bool on[V];
    const char *px[V], *pd[V];
    char* po[V];
    Vec w[V], dw[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int side = v < VQ ? side_q : 1;
        const RopeSide& s = a.side[side];
        const int first = piece * a.part_heads[side], last = min(s.heads, first + a.part_heads[side]);
        head[v] = first + (t + (v < VQ ? v : v - VQ) * team_size) / G;
        on[v] = head[v] < last && lane * 8 < D;
        if (!on[v]) head[v] = 0;
        px[v] = static_cast<const char*>(s.x) + (s.sx.row(b0, l0, head[v]) + c0) * static_cast<int>(sizeof(TX));
        pd[v] = static_cast<const char*>(s.d) + (s.sd.row(b0, l0, head[v]) + c0) * static_cast<int>(sizeof(TO));
        po[v] = static_cast<char*>(s.out) + (s.so.row(b0, l0, head[v]) + c0) * static_cast<int>(sizeof(TW));
        if (!on[v])
            for (int r = 0; r < R; ++r) ring.clear((r * V + v) * ONE, ONE);
        w[v] = vec_of(1.f);
        dw[v] = vec_of(0.f);
        if (on[v] && norm) w[v] = load_any<SPLIT>(s.weight, (norm == kQkNormToken ? head[v] * D : 0) + c0, a.w_dtype, 1.f, gap);
    }
    const RopeSide& sq = a.side[side_q];
    const RopeSide& sk = a.side[1];

    Feed feed(n, l0, a.tokens);
    auto prefetch = [&]() {
#pragma unroll
        for (int r = 0; r < R; ++r)
            feed.row([&]() {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    if (!on[v]) continue;
                    if (need_x) ring.copy<SPLIT>((r * V + v) * ONE, reinterpret_cast<const TX*>(px[v]), gap);
                    if (BWD) ring.copy<SPLIT>((r * V + v) * ONE + UX, reinterpret_cast<const TO*>(pd[v]), gap);
                }
            }, [&]() {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    px[v] += v < VQ ? sq.next_x : sk.next_x;
                    if (BWD) pd[v] += v < VQ ? sq.next_d : sk.next_d;
                }
            }, [&]() {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    px[v] += v < VQ ? sq.wrap_x : sk.wrap_x;
                    if (BWD) pd[v] += v < VQ ? sq.wrap_d : sk.wrap_d;
                }
            });
        ring.filled();
        async_commit();
    };
    for (int s = 0; s < a.stages - 1; ++s) prefetch();

    // Tables of a step's tokens (`count` of them from token tl of sample tb on), in half `which` of the team's
    // tables.
    int tb = b0, tl = l0;
    auto fill = [&](int which, int count) {
        for (int i = t; i < R * pairs; i += team_size) {
            const int r = R > 1 && i >= pairs ? 1 : 0, j = i - r * pairs, ax = axis[j];
            if (r >= count) break;
            const bool over = tl + r >= a.tokens;  // the next sample's first token
            const unsigned token = over ? 0 : tl + r;
            int p;
            if (a.positions) {
                p = a.positions[(over ? tb + 1 : tb) * a.positions_b + token * 3ll + ax];
            } else {
                const unsigned place = a.first + token, y = place / a.W, z = y / a.H;
                p = ax == 0 ? z : ax == 1 ? y - z * a.H : place - y * a.W;
            }
            const unsigned long long turn = static_cast<unsigned long long>(p + a.offset[ax]) * turns[j];
            float sn, c;  // of the signed fraction in half turns
            sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 0x1p-31f, &sn, &c);
            float* cs = table + (which * R + r) * 2 * pairs;
            if (!ALL && turns[j] == 0) c = kUnrotated;
            cs[j] = c;
            cs[pairs + j] = BWD ? -sn : sn;  // the gradient turns back
        }
        for (tl += R; tl >= a.tokens; tl -= a.tokens) ++tb;
    };
    if (n > 0) fill(0, n);
    team.sync();

    auto turn = [&](Vec& v, int r, const float2 (&c)[R][2], const float2 (&sn)[R][2]) {
        if (ALL) rotate<HALVES>(v, c[r], sn[r]);
        else if (a.rotated == kRopeSome) rotate_some<HALVES>(v, c[r], sn[r]);
    };

    const float inv_head = 1.0f / D;
    const float inv_q = 1.0f / (static_cast<float>(D) * a.side[side_q].heads);
    const float inv_k = 1.0f / (static_cast<float>(D) * max(1, a.side[1].heads));
    const int place = lane * 8 < D ? lane : 0;  // in the tables; a thread without elements reads any
    Feed store(n, l0, a.tokens);
    int which = 0;
    for (int i = 0; i < longest; i += R) {
        prefetch();
        float2 c[R][2], sn[R][2];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float* cs = table + (which * R + r) * 2 * pairs;
            if constexpr (SPLIT && !HALVES) {  // two pairs of each half
                const float2* t2 = reinterpret_cast<const float2*>(cs);
                c[r][0] = t2[place], c[r][1] = t2[pairs / 4 + place];
                sn[r][0] = t2[pairs / 2 + place], sn[r][1] = t2[pairs / 2 + pairs / 4 + place];
            } else {
                const float4 u = reinterpret_cast<const float4*>(cs)[place], z = reinterpret_cast<const float4*>(cs + pairs)[place];
                c[r][0] = make_float2(u.x, u.y), c[r][1] = make_float2(u.z, u.w);
                sn[r][0] = make_float2(z.x, z.y), sn[r][1] = make_float2(z.z, z.w);
            }
        }
        which ^= 1;
        if (i + R < n) fill(which, n - i - R);
        // every thread has read this step's tables and sees the next ones after a barrier of the team
        if (!WIDE || norm != kQkNormToken) team.sync();
        ring_wait(a.stages);

        Vec x[R][V], g[R][V];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                if (need_x) x[r][v] = ring.read<TX>((r * V + v) * ONE);
                if (BWD) {
                    g[r][v] = ring.read<TO>((r * V + v) * ONE + UX);
                    turn(g[r][v], r, c, sn);
                }
            }
        ring.done();
        // per vector: rd = 1 / rms, and rd^2 mean(g w x) of the norm it belongs to
        float rd[R][V], gx[R][V];
        if (norm) {
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const Vec& xv = x[r][v];
                    float2 s1 = mul2(xv.f[0], xv.f[0]), s2 = both(0.f);
#pragma unroll
                    for (int e = 1; e < 4; ++e) s1 = fma2(xv.f[e], xv.f[e], s1);
                    if (BWD)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s2 = fma2(mul2(g[r][v].f[e], w[v].f[e]), xv.f[e], s2);
                    rd[r][v] = fold(s1);
                    gx[r][v] = BWD ? fold(s2) : 0.f;
                }
            if (norm == kQkNormHead) {
                for (int o = G >> 1; o > 0; o >>= 1)
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            rd[r][v] += Team<WIDE>::swap(rd[r][v], o);
                            if (BWD) gx[r][v] += Team<WIDE>::swap(gx[r][v], o);
                        }
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        rd[r][v] = rsqrtf(rd[r][v] * inv_head + a.eps);
                        gx[r][v] *= inv_head * rd[r][v] * rd[r][v];
                    }
            } else {
                constexpr int S = VK ? 2 : 1, N = S * (BWD ? 2 : 1);  // sums of a row: x^2 a side, then g w x
                float sums[N * R];
#pragma unroll
                for (int r = 0; r < R; ++r) {
#pragma unroll
                    for (int i = 0; i < N; ++i) sums[N * r + i] = 0.f;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const int side = v < VQ ? 0 : S - 1;
                        sums[N * r + side] += rd[r][v];
                        if constexpr (BWD) sums[N * r + S + side] += gx[r][v];
                    }
                }
                team.sum(sums);
#pragma unroll
                for (int r = 0; r < R; ++r)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const int side = v < VQ ? 0 : S - 1;
                        const float inv = side == 0 ? inv_q : inv_k;
                        rd[r][v] = rsqrtf(sums[N * r + side] * inv + a.eps);
                        if constexpr (BWD) gx[r][v] = sums[N * r + S + side] * inv * rd[r][v] * rd[r][v];
                    }
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            store.row([&]() {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    TW* out = reinterpret_cast<TW*>(po[v]);
                    if (!BWD) {
                        if (norm)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[r][v].f[e] = mul2(x[r][v].f[e], mul2(w[v].f[e], both(rd[r][v])));
                        turn(x[r][v], r, c, sn);
                        if (on[v]) store_vec<TW, SPLIT>(out, x[r][v], gap);
                    } else {
                        if (norm) {
                            const float2 rr = both(rd[r][v]), mg = both(-gx[r][v]);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                dw[v].f[e] = fma2(g[r][v].f[e], mul2(x[r][v].f[e], rr), dw[v].f[e]);
                                g[r][v].f[e] = mul2(rr, fma2(x[r][v].f[e], mg, mul2(g[r][v].f[e], w[v].f[e])));
                            }
                        }
                        if (on[v]) store_vec<TW, SPLIT>(out, g[r][v], gap);
                    }
                }
            }, [&]() {
#pragma unroll
                for (int v = 0; v < V; ++v) po[v] += v < VQ ? sq.next_o : sk.next_o;
            }, [&]() {
#pragma unroll
                for (int v = 0; v < V; ++v) po[v] += v < VQ ? sq.wrap_o : sk.wrap_o;
            });
        }
    }

    if (!BWD || !a.part) return;
    launch_dependents();
    const int sides = a.side[1].heads > 0 ? 2 : 1;
    if (norm == kQkNormToken) {
        float* sums = a.part + static_cast<long long>(worker) * (a.side[0].heads + a.side[1].heads) * D + c0;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (on[v])
                store_vec<float, SPLIT>(sums + (head[v] + ((v < VQ ? side_q : 1) ? a.side[0].heads : 0)) * D, dw[v], gap);
        return;
    }
    // one weight for all heads of a side: joined over the block's heads in order, through the ring's memory
    async_wait<0>();
    __syncthreads();
    Vec* sums = reinterpret_cast<Vec*>(shared);
#pragma unroll
    for (int v = 0; v < V; ++v) sums[v * blockDim.x + threadIdx.x] = dw[v];
    __syncthreads();
    for (int j = t; j < sides * G; j += team_size) {
        const int side = j / G, place = j % G;
        if (place * 8 >= D) continue;
        Vec d = vec_of(0.f);
        // none where the other blocks have this side
        const int count = a.split_sides && side != part ? 0 : min(a.side[side].heads - piece * a.part_heads[side], a.part_heads[side]);
        for (int h = 0; h < count; ++h) {
            const int slot = h * G + place, v = slot / team_size + (side != side_q ? VQ : 0);
            const Vec u = sums[v * blockDim.x + in_block * team_size + slot % team_size];
#pragma unroll
            for (int e = 0; e < 4; ++e) d.f[e] = add2(d.f[e], u.f[e]);
        }
        store_vec<float, SPLIT>(a.part + ((static_cast<long long>(worker) * a.parts + part) * sides + side) * D + place * (SPLIT ? 4 : 8), d, gap);
    }
}

// Registers of a thread with V vectors (block-wide teams, several teams a block), and the blocks that an SM
// then holds at once.  Without a norm the backward is a rotation alone.
inline int rope_blocks_per_sm(const RowPlan& p, bool backward, bool norm) {
    const int wide[3][4] = {{0, 80, 96, 128}, {0, 96, 120, 168}, {0, 48, 64, 64}};
    const int narrow[3][3] = {{0, 80, 120}, {0, 128, 136}, {0, 64, 64}};
    const int kind = !backward ? 0 : norm ? 1 : 2;
    // a quarter of the registers and of the warps each to an SM's four parts
    const int warps = 4 * (16384 / (32 * (p.team <= 32 ? narrow[kind][p.V] : wide[kind][p.V])));
    return std::max(1, warps * 32 / p.threads);
}

template <typename TX, typename TO, int VQ, int VK, bool HALVES, bool BWD, bool WIDE, int NORM, bool ALL>
cudaError_t rope_launch(QkRopeArgs a, const RowPlan& p, cudaStream_t st) {
    for (RopeSide& s : a.side) {
        const long long x = sizeof(TX), d = sizeof(TO), o = BWD ? sizeof(TX) : sizeof(TO);
        s.next_x = s.sx.l * x, s.wrap_x = (s.sx.b - a.tokens * s.sx.l) * x;
        s.next_d = s.sd.l * d, s.wrap_d = (s.sd.b - a.tokens * s.sd.l) * d;
        s.next_o = s.so.l * o, s.wrap_o = (s.so.b - a.tokens * s.so.l) * o;
    }
    constexpr int R = kRows<VQ + VK, BWD>;
    const size_t stage = size_t(16) * R * (VQ + VK) * (kUnits<TX> + (BWD ? kUnits<TO> : 0)) * p.threads;
    const int per_sm = rope_blocks_per_sm(p, BWD, a.norm != kQkNormNone);
    a.stages = ring_stages(stage, per_sm, kRopeRingBytes / per_sm, a.share, R);
    const size_t smem = a.stages * stage + size_t(p.threads / p.team) * 2 * R * a.head_dim * sizeof(float);
    const auto kernel = qk_rope_kernel<TX, TO, VQ, VK, HALVES, BWD, WIDE, NORM, ALL>;
    const cudaError_t e = allow_shared(kernel, smem, kRopeRingBytes + kRopeTableBytes);
    if (e != cudaSuccess) return e;
    kernel<<<p.blocks, p.threads, smem, st>>>(a);
    return cudaGetLastError();
}
template <typename TX, typename TO, bool BWD, int NORM, bool ALL>
cudaError_t rope_launch_types(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st) {
    const auto shape = [&](auto vq, auto vk, auto wide) {
        constexpr int VQ = decltype(vq)::value, VK = decltype(vk)::value;
        constexpr bool WIDE = decltype(wide)::value;
        return a.halves ? rope_launch<TX, TO, VQ, VK, true, BWD, WIDE, NORM, ALL>(a, p, st)
                        : rope_launch<TX, TO, VQ, VK, false, BWD, WIDE, NORM, ALL>(a, p, st);
    };
    const std::integral_constant<int, 0> none;
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 2> two;
    const bool k = p.V > p.VQ;
    if (p.team <= 32) return k ? shape(one, one, std::false_type()) : shape(one, none, std::false_type());
    if (p.VQ == 1) return k ? shape(one, one, std::true_type()) : shape(one, none, std::true_type());
    return k ? shape(two, one, std::true_type()) : shape(two, none, std::true_type());
}

// The kernels of one direction and norm (NORM -1: any), for calls that rotate every pair (ALL) and for the others,
// each in a file of its own.
template <bool BWD, int NORM, bool ALL>
cudaError_t rope_launch_all(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st) {
    if (a.x_dtype == kF32) return rope_launch_types<float, float, BWD, NORM, ALL>(a, p, st);
    if (a.x_dtype == kBf16)
        return a.out_dtype == kF32 ? rope_launch_types<__nv_bfloat16, float, BWD, NORM, ALL>(a, p, st)
                                   : rope_launch_types<__nv_bfloat16, __nv_bfloat16, BWD, NORM, ALL>(a, p, st);
    return a.out_dtype == kF32 ? rope_launch_types<__half, float, BWD, NORM, ALL>(a, p, st)
                               : rope_launch_types<__half, __half, BWD, NORM, ALL>(a, p, st);
}
cudaError_t launch_qk_rope_fwd(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st);
cudaError_t launch_qk_rope_bwd_none(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st);
cudaError_t launch_qk_rope_bwd_head(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st);
cudaError_t launch_qk_rope_bwd_token(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st);
cudaError_t launch_qk_rope_fwd_some(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st);
cudaError_t launch_qk_rope_bwd_none_some(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st);
cudaError_t launch_qk_rope_bwd_head_some(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st);
cudaError_t launch_qk_rope_bwd_token_some(const QkRopeArgs& a, const RowPlan& p, cudaStream_t st);

}  // namespace slra
